"""Refusals of slim_dequant_grouped_gemm and slim_token_logprobs: checked on the
host before any device work, at the C entry points and in the binding."""
import pytest
import torch

from post_weight_quantization_hessian_b200 import build, slim

EINVAL = 1


@pytest.fixture(scope="module")
def lib():
    build.build()
    return slim._lib()


def grouped(lib, **kw):
    a = dict(codes=0x1000, bits=0x2000, scale=0x3000, zero=0x4000, E=4, m=256, n=640, group=128, avg=2, x=0x5000, xd=1,
             T=100, index=None, offsets=0x6000, R=100, y=0x7000, yd=1, ws=None, wsb=0)
    a.update(kw)
    return lib.slim_dequant_grouped_gemm(*[a[k] for k in ("codes", "bits", "scale", "zero", "E", "m", "n", "group",
                                                          "avg", "x", "xd", "T", "index", "offsets", "R", "y", "yd",
                                                          "ws", "wsb")], None)


@pytest.mark.parametrize("kw, why", [
    (dict(E=0), "no expert"),
    (dict(E=1025), "too many experts"),
    (dict(group=96), "group not in {32, 64, 128}"),
    (dict(n=640 + 32), "n % group != 0"),
    (dict(m=0), "no output"),
    (dict(avg=1), "avg_bits below 2"),
    (dict(avg=8), "avg_bits above 7"),
    (dict(R=-1), "negative row count"),
    (dict(R=2 ** 29 + 1, T=2 ** 30), "too many rows"),
    (dict(E=1024, m=2 ** 21), "E m past 31 bits"),
    (dict(T=99), "fewer rows of x than grouped rows, and no index"),
    (dict(T=-1, index=0x8000), "negative T"),
    (dict(xd=2), "unknown x dtype"),
    (dict(yd=2), "unknown y dtype"),
    (dict(codes=None), "NULL codes"),
    (dict(bits=None), "NULL bits"),
    (dict(scale=None), "NULL scale"),
    (dict(zero=None), "NULL zero"),
    (dict(x=None), "NULL x"),
    (dict(offsets=None), "NULL offsets"),
    (dict(y=None), "NULL y"),
    (dict(codes=0x1004), "codes not 16-byte aligned"),
    (dict(x=0x5008), "x not 16-byte aligned"),
    (dict(y=0x7001), "y not aligned to bf16"),
    (dict(y=0x7002, yd=0), "y not aligned to float32"),
    (dict(index=0x8002), "row_index not aligned"),
    (dict(offsets=0x6001), "offsets not aligned"),
])
def test_grouped_refusals(lib, kw, why):
    assert grouped(lib, **kw) == EINVAL, why


def test_grouped_of_no_rows_is_ok_without_a_device(lib):
    assert grouped(lib, R=0, T=0) == 0
    assert lib.slim_dequant_grouped_gemm_workspace_bytes(4, 256, 641, 128, 2, 1, 1, 100) == 0
    assert lib.slim_dequant_grouped_gemm_workspace_bytes(4, 256, 640, 96, 2, 1, 0, 100) == 0   # not a valid call


@pytest.mark.parametrize("kw, why", [
    (dict(dtype=3), "unknown dtype"),
    (dict(N=-1), "negative row count"),
    (dict(V=0), "empty vocabulary"),
    (dict(V=2 ** 31, ld=2 ** 31), "vocabulary past 31 bits"),
    (dict(ld=999), "rows overlap"),
    (dict(k=33, tl=0x5000, ti=0x6000), "top_k above 32"),
    (dict(k=-1), "negative top_k"),
    (dict(V=4, ld=4, k=5, tl=0x5000, ti=0x6000), "top_k above V"),
    (dict(k=2), "NULL top outputs"),
    (dict(k=2, tl=0x5000), "NULL top_id"),
    (dict(tl=0x5000, ti=0x6000), "top outputs without top_k"),
    (dict(logits=None), "NULL logits"),
    (dict(logits=0x1002), "float32 logits not aligned"),
    (dict(tokens=0x2004), "tokens not aligned"),
    (dict(logp=0x3002), "logp not aligned"),
])
def test_logprobs_refusals(lib, kw, why):
    a = dict(logits=0x1000, dtype=0, N=4, V=1000, ld=1000, tokens=0x2000, k=0, logp=0x3000, ent=0x4000, tl=None, ti=None)
    a.update(kw)
    rc = lib.slim_token_logprobs(a["logits"], a["dtype"], a["N"], a["V"], a["ld"], a["tokens"], a["k"], a["logp"],
                                 a["ent"], a["tl"], a["ti"], None)
    assert rc == EINVAL, why


def test_logprobs_of_no_rows_is_ok_without_a_device(lib):
    assert lib.slim_token_logprobs(None, 0, 0, 1000, 1000, None, 0, None, None, None, None, None) == 0
    assert lib.slim_token_logprobs(None, 0, 0, 1000, 1000, None, 5, None, None, None, None, None) == 0


def binding_args(**kw):
    a = dict(codes=torch.zeros((2, 8, 16), dtype=torch.int32), bits=torch.full((2, 2), 2, dtype=torch.uint8),
             scale=torch.ones((2, 8, 2)), zero=torch.ones((2, 8, 2)), group=128, avg_bits=2,
             x=torch.zeros((5, 256), dtype=torch.bfloat16), offsets=torch.zeros(3, dtype=torch.int32))
    a.update(kw)
    return a


@pytest.mark.parametrize("kw", [
    dict(x=torch.zeros((5, 128))),
    dict(x=torch.zeros((5, 256), dtype=torch.float16)),
    dict(codes=torch.zeros((2, 8, 8), dtype=torch.int32)),
    dict(bits=torch.full((2, 2), 2)),
    dict(zero=torch.ones((2, 8, 2), dtype=torch.float64)),
    dict(offsets=torch.zeros(3, dtype=torch.int64)),
    dict(offsets=torch.zeros(4, dtype=torch.int32)),
    dict(row_index=torch.zeros(5, dtype=torch.int64)),
    dict(y=torch.zeros((5, 7))),
    dict(y=torch.zeros((5, 8)), y_dtype=torch.bfloat16),
    dict(y_dtype=torch.float16),
    dict(),                                   # CPU tensors
])
def test_grouped_binding_refusals(kw):
    with pytest.raises(ValueError):
        slim.slim_dequant_grouped_gemm(**binding_args(**kw))


@pytest.mark.parametrize("logits, kw", [
    (torch.zeros(8), {}),
    (torch.zeros((2, 8), dtype=torch.float16), {}),
    (torch.zeros((8, 2)).t(), {}),
    (torch.zeros((1, 8)).expand(2, 8), {}),
    (torch.zeros((2, 8)), dict(top_k=9)),
    (torch.zeros((2, 40)), dict(top_k=33)),
    (torch.zeros((2, 8)), dict(tokens=torch.zeros(2, dtype=torch.int32))),
    (torch.zeros((2, 8)), dict(tokens=torch.zeros(3, dtype=torch.int64))),
    (torch.zeros((2, 8)), {}),                # CPU tensors
])
def test_logprobs_binding_refusals(logits, kw):
    with pytest.raises(ValueError):
        slim.slim_token_logprobs(logits, **kw)
