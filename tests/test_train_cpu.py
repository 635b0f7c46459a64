"""Argument checks and workspace sizes of the training-step operators (no GPU:
every refusal comes before anything touches a device)."""

import pytest

from double_binary_tree_amd import emucomm as E

A = 1 << 20                         # pointers far apart, never followed
P = [A * (k + 1) for k in range(64)]
F32, F16, BF16, I32 = (E.DTYPE[k] for k in ("f32", "f16", "bf16", "i32"))
BAD = E.ERR_INVALID_ARGUMENT


def loss(vocab=(10, 6), tokens=4, dim=16, dtype=F32, x=P[0], w=(P[1], P[2]), y=P[3], out=P[4], lse=P[5], ws=P[6],
         size=1 << 19):
    return E.cross_entropy_raw(x, w, vocab, y, tokens, dim, out, lse, dtype, ws, size)


def grad(vocab=(10, 6), tokens=4, dim=16, dtype=F32, x=P[0], w=(P[1], P[2]), y=P[3], lse=P[4], d=P[5], dx=P[6],
         dw=(P[7], P[8]), ws=P[9], size=1 << 19):
    return E.cross_entropy_grad_raw(x, w, vocab, y, lse, d, tokens, dim, dx, dw, dtype, ws, size)


@pytest.mark.parametrize("change", [
    {"dtype": I32}, {"dtype": 9}, {"vocab": ()}, {"vocab": (0, 0)}, {"dim": 0}, {"dim": 17}, {"dim": 18}, {"dim": 1 << 17},
    {"dim": 12, "dtype": F16}, {"dim": 12, "dtype": BF16}, {"tokens": (1 << 20) + 1}, {"vocab": ((1 << 24) + 1, 6)},
    {"vocab": (1 << 23, (1 << 23) + 1)}, {"vocab": (1 << 18, 0), "tokens": (1 << 20)}, {"vocab": (1 << 15, 1), "tokens": (1 << 20)}, {"x": None}, {"x": A + 4}, {"w": None},
    {"w": (P[1], None)}, {"w": (P[1] + 8, P[2])}, {"y": None}, {"y": P[3] + 8}, {"lse": None}, {"ws": None},
    {"ws": P[6] + 8}, {"size": 0}, {"ws": P[1]}, {"vocab": (1,) * 65, "w": (P[1],) * 65}])
def test_cross_entropy_refuses(change):
    assert loss(**change) == BAD
    assert grad(**change) == BAD


@pytest.mark.parametrize("change", [{"out": None}, {"out": P[4] + 4}, {"out": P[5]}, {"out": P[3]}, {"lse": P[0]}])
def test_cross_entropy_refuses_outputs(change):
    assert loss(**change) == BAD


@pytest.mark.parametrize("change", [{"dx": None, "dw": None}, {"dx": P[6] + 8}, {"dx": P[0]}, {"dw": (P[7], None)},
                                    {"dw": (P[7], P[7])}, {"dw": (P[1], P[8])}, {"d": None}, {"d": P[5] + 4}])
def test_cross_entropy_grad_refuses(change):
    assert grad(**change) == BAD


def test_cross_entropy_workspace_sizes():
    for dims in ((0, 0), (1, 0), (0, 1), (1, 1)):
        e, n = E.cross_entropy_workspace_raw((50000, 50257), 4096, 2048, BF16, *dims)
        assert e == 0 and n > 0
        # far below the logits, which are not kept (one f32 logit per token and row)
        assert n < 4096 * 100257 * 4 // 2 + (1 << 30)
    assert E.cross_entropy_workspace_raw((10,), 0, 16, F32, 0, 0) == (0, 0)
    e, small = E.cross_entropy_workspace_raw((10, 6), 4, 16, F32, 0, 0)
    assert e == 0 and loss(size=small - 1) == BAD
    e, small = E.cross_entropy_workspace_raw((10, 6), 4, 16, F32, 1, 1)
    assert e == 0 and grad(size=small - 1) == BAD
    assert E.cross_entropy_workspace_raw((10,), 4, 17, F32, 0, 0)[0] == BAD
    assert E.cross_entropy_workspace_raw((10,), 4, 16, I32, 0, 0)[0] == BAD
    assert E.lib().emu_cross_entropy_workspace(1, None, 4, 16, F32, 0, 0, None) == BAD


def test_no_tokens_need_no_buffers():
    assert loss(tokens=0, x=None, y=None, out=None, lse=None, ws=None, size=0) == E.SUCCESS
    assert grad(tokens=0, x=None, y=None, lse=None, d=None, dx=None, dw=None, ws=None, size=0) == BAD
    assert grad(tokens=0, x=None, y=None, lse=None, d=None, dx=P[6], dw=None, ws=None, size=0) == E.SUCCESS


def balance(logits=(P[0], P[1]), experts=(P[2], P[3]), tokens=(5, 7), nexp=8, topk=2, coef=0.1, counts=P[4], out=P[5],
            dz=(P[6], P[7]), dtype=F32, ws=P[8], size=1 << 19):
    return E.balance_loss_raw(logits, experts, tokens, nexp, topk, coef, counts, out, dz, dtype, ws, size)


@pytest.mark.parametrize("change", [
    {"dtype": I32}, {"tokens": ()}, {"tokens": (5, (1 << 24) + 1)}, {"nexp": 0}, {"nexp": 1025}, {"topk": 0}, {"topk": 9},
    {"coef": float("nan")}, {"coef": float("inf")}, {"logits": None}, {"logits": (P[0], None)}, {"logits": (P[0] + 4, P[1])},
    {"experts": None}, {"experts": (P[2], None)}, {"experts": (P[2], P[3] + 4)}, {"counts": None}, {"counts": P[4] + 8},
    {"out": None}, {"out": P[5] + 4}, {"dz": (P[6], None)}, {"dz": (P[6], P[6])}, {"dz": (P[0], P[7])}, {"ws": None},
    {"ws": P[8] + 8}, {"ws": P[2]}, {"size": 0}, {"counts": P[0]}, {"out": P[4]}, {"tokens": (1,) * 65}])
def test_balance_loss_refuses(change):
    assert balance(**change) == BAD


def test_balance_loss_workspace_sizes():
    e, n = E.balance_loss_workspace_raw((5, 7), 8)
    assert e == 0 and n > 0 and balance(size=n - 1) == BAD
    assert E.balance_loss_workspace_raw((0, 0), 8)[0] == 0
    assert E.balance_loss_workspace_raw((5,), 0)[0] == BAD
    assert E.lib().emu_balance_loss_workspace(1, None, 8, None) == BAD


def ortho(sends=(P[0], P[1]), recvs=(P[2], P[3]), rows=8, cols=12, steps=5, coeffs=None, dtype=F32, ws=P[4],
          size=1 << 19):
    return E.orthogonalize_raw(sends, recvs, rows, cols, steps, coeffs, dtype, ws, size)


@pytest.mark.parametrize("change", [
    {"dtype": I32}, {"sends": ()}, {"sends": None, "recvs": ()}, {"sends": (P[0], None)}, {"sends": (P[0] + 8, P[1])}, {"recvs": None},
    {"recvs": (P[2], None)}, {"recvs": (P[2], P[3] + 4)}, {"recvs": (P[2], P[2])}, {"recvs": (P[1], P[3])},
    {"rows": (1 << 20) + 1}, {"cols": (1 << 20) + 1}, {"rows": 1 << 20, "cols": 1 << 13}, {"steps": 0}, {"steps": 17}, {"steps": -1},
    {"coeffs": [1.0, 2.0, float("nan")] * 5}, {"coeffs": [float("inf")] * 15}, {"ws": None}, {"ws": P[4] + 8}, {"ws": P[0]},
    {"size": 0}, {"sends": (P[0],) * 65, "recvs": (P[2],) * 65}])
def test_orthogonalize_refuses(change):
    if change.get("sends", 0) is None:
        assert E.lib().emu_orthogonalize(2, None, None, 8, 12, 5, None, F32, P[4], 1 << 19, None) == BAD
        return
    assert ortho(**change) == BAD


def test_orthogonalize_workspace_sizes():
    e, n = E.orthogonalize_workspace_raw(2, 8, 12, F32)
    assert e == 0 and n > 0 and ortho(size=n - 1) == BAD
    assert E.orthogonalize_workspace_raw(2, 0, 12, F32) == (0, 0)
    assert ortho(rows=0, sends=(None, None), recvs=(None, None), ws=None, size=0) == E.SUCCESS
    assert E.orthogonalize_workspace_raw(0, 8, 12, F32)[0] == BAD
    assert E.orthogonalize_workspace_raw(2, 8, 12, I32)[0] == BAD
    assert E.lib().emu_orthogonalize_workspace(2, 8, 12, F32, None) == BAD


def test_tensor_calls_refuse_cpu_tensors():
    import torch
    x, w, y = torch.zeros(4, 16), torch.zeros(8, 16), torch.zeros(4, dtype=torch.int64)
    f, e = torch.zeros(4), torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: E.cross_entropy_tensors(x, [w], y, f, f.clone()),
                 lambda: E.cross_entropy_grad_tensors(x, [w], y, f, f, torch.zeros_like(x), [torch.zeros_like(w)]),
                 lambda: E.balance_loss_tensors([x], [e], 0.1, torch.zeros(2, 16, dtype=torch.int64), f[:1]),
                 lambda: E.orthogonalize_tensors([x], [x]), lambda: E.orthogonalize_tensors([], [])):
        with pytest.raises(ValueError):
            call()
