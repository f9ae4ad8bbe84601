"""What the 16-bit products refuse, without a GPU: the argument checks run before any device access
(addresses here are made up and never read)."""
import pytest
import torch

import quantized_moe_routed_amd as moe
from quantized_moe_routed_amd import GroupsDesc, Mat, dense

P = 1 << 20      # an aligned address


def mat(ld, dt=moe.T_BF16, rows=0, p=P):
    return Mat(p, ld, dt, rows)


def gdesc(T=4, k=2, E=8, E_local=8, offsets=P, slots=P, g2l=None):
    return GroupsDesc(offsets, slots, g2l, T, k, E, E_local)


def refused(status, text, f, *a):
    with pytest.raises(moe.MoeError) as e:
        f(*a, 0)
    assert e.value.status == status and text in str(e.value), str(e.value)


ARG, UNSUP, WS = moe.ERR_ARG, moe.ERR_UNSUPPORTED, moe.ERR_WORKSPACE


@pytest.mark.parametrize("change,status,text", [
    (dict(N=12), ARG, "N = 12"),
    (dict(K=0), ARG, "K = 0"),
    (dict(K=1 << 21), UNSUP, "K = 2097152"),
    (dict(x=None), ARG, "x must not be NULL"),
    (dict(x=mat(64, p=None)), ARG, "x must not be NULL"),
    (dict(x=mat(64, moe.T_F32)), UNSUP, "bf16 or fp16"),
    (dict(x=mat(64, 9)), UNSUP, "bf16 or fp16"),
    (dict(x=mat(56)), ARG, "row stride 56"),
    (dict(x=mat(68)), ARG, "multiples of 16 bytes"),
    (dict(x=mat(64, p=P + 8)), ARG, "multiples of 16 bytes"),
    (dict(x=mat(64, rows=3)), ARG, "row order 3"),
    (dict(w=None), ARG, "w must not be NULL"),
    (dict(w=P + 2), ARG, "16-byte aligned"),
    (dict(y=mat(32, moe.T_F16)), UNSUP, "y has type 2"),
    (dict(y=mat(32, rows=moe.ROWS_TOKEN)), ARG, "y: row order 2"),
    (dict(g=None), ARG, "groups is NULL"),
    (dict(g=gdesc(T=-1)), ARG, "T = -1"),
    (dict(g=gdesc(k=0)), ARG, "k = 0"),
    (dict(g=gdesc(E=2000, E_local=2000)), UNSUP, "E = 2000"),
    (dict(g=gdesc(E_local=9)), ARG, "E_local = 9"),
    (dict(g=gdesc(E_local=4)), ARG, "E_local = 4 without g2l"),
    (dict(g=gdesc(T=1 << 29, k=4)), UNSUP, "T * k"),
    (dict(g=gdesc(offsets=None)), ARG, "offsets"),
    (dict(g=gdesc(slots=None), x=mat(64, rows=moe.ROWS_TOKEN)), ARG, "needs slot_list"),
])
def test_grouped_matmul_refuses(change, status, text):
    a = dict(x=mat(64), w=P, N=32, K=64, g=gdesc(), y=mat(32))
    a.update(change)
    refused(status, text, moe.grouped_matmul, a["x"], a["w"], a["N"], a["K"], a["g"], a["y"])


def test_made_up_addresses_are_no_device_memory():
    refused(moe.ERR_HIP if not torch.cuda.is_available() else moe.ERR_DEVICE, "", moe.grouped_matmul, mat(64), P, 32,
            64, gdesc(), mat(32))


def test_empty_batches_are_no_ops():
    moe.grouped_matmul(None, None, 32, 64, gdesc(T=0), None, 0)
    moe.grouped_swiglu(None, None, None, 32, 64, gdesc(T=0), None, None, None, 0)
    moe.grouped_matmul_grad(None, None, None, 32, 64, gdesc(T=0), None, None, 0, 1, 0)
    moe.linear(None, None, None, 0, None, 0, 32, 64, None, None, 0)
    moe.cross_entropy(None, None, None, 0, 5, 64, None, None, None, 0, 0)


@pytest.mark.parametrize("change,status,text", [
    (dict(dy=mat(24)), ARG, "dy has row stride"),
    (dict(dy=mat(32, moe.T_F16)), UNSUP, "dy has type"),
    (dict(dx=mat(64, rows=moe.ROWS_TOKEN)), ARG, "dx: row order 2"),
    (dict(dw=P, dw_dt=moe.T_F16), UNSUP, "dw has type 2"),
    (dict(dw=P + 4), ARG, "dw must be 16-byte aligned"),
])
def test_grouped_matmul_grad_refuses(change, status, text):
    a = dict(dy=mat(32), dx=mat(64), dw=P, dw_dt=moe.T_BF16)
    a.update(change)
    refused(status, text, moe.grouped_matmul_grad, a["dy"], mat(64), P, 32, 64, gdesc(), a["dx"], a["dw"], a["dw_dt"], 0)


def test_grouped_swiglu_refuses():
    refused(ARG, "up must not", moe.grouped_swiglu, mat(64), P, None, 32, 64, gdesc(), mat(32), None, None)
    refused(UNSUP, "h has type 0", moe.grouped_swiglu, mat(64), P, P, 32, 64, gdesc(), mat(32, moe.T_F32), None, None)
    refused(ARG, "keep_u must be in grouped", moe.grouped_swiglu, mat(64), P, P, 32, 64, gdesc(), mat(32), None,
            mat(32, rows=1))
    n = moe.grouped_swiglu_grad_workspace(4, 2, 32)
    assert n >= 2 * 8 * 32 * 2
    args = [mat(32), mat(64), P, P, mat(32), mat(32), 32, 64, gdesc(), mat(64), P, P, moe.T_F32, 0]
    refused(WS, f"need {n}", moe.grouped_swiglu_grad, *args, P, n - 1)
    refused(WS, f"need {n}", moe.grouped_swiglu_grad, *args, None, n)
    refused(ARG, "go together", moe.grouped_swiglu_grad, *args[:10], None, P, moe.T_F32, 0, P, n)
    refused(ARG, "keep_g must not", moe.grouped_swiglu_grad, *args[:4], None, *args[5:], P, n)


def test_linear_refuses():
    base = dict(x=mat(64), w=P, bias=None, fn=0, res=None, T=3, N=32, K=64, y=mat(32), pre=None)
    for change, status, text in ((dict(fn=4), UNSUP, "activation 4"), (dict(T=-1), ARG, "T < 0"),
                                 (dict(bias=P + 4), ARG, "bias"), (dict(res=mat(32, moe.T_F32)), UNSUP, "residual has type"),
                                 (dict(pre=mat(32, moe.T_F32)), UNSUP, "pre has type"), (dict(N=33), ARG, "N = 33")):
        a = {**base, **change}
        refused(status, text, moe.linear, *a.values())
    n = moe.linear_grad_workspace(3, 32, 64)
    g = dict(dy=mat(32), x=mat(64), w=P, pre=None, fn=2, T=3, N=32, K=64, dx=mat(64), dw=P, dw_dt=1, dbias=P, acc=0,
             ws=P, n=n)
    for change, status, text in ((dict(), ARG, "pre must not be NULL"), (dict(fn=0, n=n - 1), WS, "workspace"),
                                 (dict(fn=0, dbias=P + 8), ARG, "dbias"), (dict(fn=0, dw_dt=2), UNSUP, "dw has type")):
        a = {**g, **change}
        refused(status, text, moe.linear_grad, *a.values())


def test_cross_entropy_refuses():
    f, b = moe.cross_entropy_workspace(5, 100, 64)
    base = dict(x=mat(64), w=P, t=P, T=5, V=100, H=64, nll=P, lse=P, ws=P, n=f)
    for change, status, text in ((dict(V=0), ARG, "V = 0"), (dict(H=60), ARG, "H = 60"), (dict(t=None), ARG, "target"),
                                 (dict(nll=None), ARG, "nll and lse"), (dict(n=f - 1), WS, f"need {f}")):
        a = {**base, **change}
        refused(status, text, moe.cross_entropy, *a.values())
    g = dict(x=mat(64), w=P, t=P, lse=P, dnll=P, T=5, V=100, H=64, dx=mat(64), dw=P, dt=1, acc=0, ws=P, n=b)
    for change, status, text in ((dict(lse=None), ARG, "lse and dnll"), (dict(dx=mat(56)), ARG, "dx has row stride"),
                                 (dict(dt=2), UNSUP, "dw has type"), (dict(n=b - 1), WS, f"need {b}")):
        a = {**g, **change}
        refused(status, text, moe.cross_entropy_grad, *a.values())


def test_python_calls_check_their_tensors():
    bf = torch.bfloat16
    x, w = torch.zeros((3, 64), dtype=bf), torch.zeros((32, 64), dtype=bf)
    off, slots = torch.zeros(5, dtype=torch.int32), torch.zeros(6, dtype=torch.int32)
    g = dense.Groups(off, slots, 3, 2)
    assert (g.E, g.E_local, g.slots) == (4, 4, 6)
    with pytest.raises(ValueError, match="slot_list holds 6"):
        dense.Groups(off, slots, 4, 2)
    with pytest.raises(ValueError, match="offsets"):
        dense.Groups(off.long(), slots, 3, 2)
    with pytest.raises(ValueError, match="w must be"):
        dense.linear(x, w.half())
    with pytest.raises(ValueError, match="w must be"):
        dense.linear(x, torch.zeros((64, 32), dtype=bf).t())
    with pytest.raises(ValueError, match="residual has shape"):
        dense.linear(x, w, residual=x)
    with pytest.raises(ValueError, match="activation 'tanh'"):
        dense.linear(x, w, act="tanh")
    with pytest.raises(ValueError, match="rows of x must be contiguous"):
        dense.linear(torch.zeros((64, 3), dtype=bf).t(), w)
    with pytest.raises(TypeError, match="float64"):
        dense.linear(x.double(), w.double())
    with pytest.raises(ValueError, match="accumulate needs"):
        dense.linear_grad(torch.zeros((3, 32), dtype=bf), x, w, accumulate=True)
    with pytest.raises(ValueError, match="target must be"):
        dense.cross_entropy(x, w, torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="expected \\(6, 64\\)"):
        dense.grouped_matmul(x, torch.zeros((4, 32, 64), dtype=bf), g)
