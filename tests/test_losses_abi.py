"""The losses' argument checks, made without a GPU: every refused call names its
fault and enqueues nothing."""

import ctypes

import pytest

from tests._lib import load

zr = load()
torch = pytest.importorskip("torch")

lib = zr._lib
A = 0x10000         # an address that no refused call reads

DISTILL = dict(logits=A, dtype=zr.ZR_FP32, rows=3, vocab=10, logits_stride=10, ids=A, ids_type=zr.ZR_I32,
               ids_stride=4, teacher=A, teacher_dtype=zr.ZR_FP32, teacher_stride=4, top=4, weight=A,
               temperature=1.0, loss=A, dlogits=A, dlogits_stride=10, workspace=None, workspace_bytes=0,
               stream=None)
POLICY = dict(logits=A, dtype=zr.ZR_BF16, rows=3, vocab=10, logits_stride=10, tokens=A, token_type=zr.ZR_I64,
              old_logp=A, ref_logp=A, advantage=A, weight=A, clip_low=0.2, clip_high=0.2, kl=0.1,
              temperature=1.0, loss=A, logp=A, dlogits=A, dlogits_stride=10, workspace=None,
              workspace_bytes=0, stream=None)
NAN = float("nan")

BOTH = [(dict(dtype=2), "dtype"), (dict(rows=-1), "rows must"), (dict(vocab=0), "vocab >= 1"),
        (dict(vocab=1 << 30, logits_stride=1 << 30, dlogits_stride=1 << 30), "2^30"),
        (dict(rows=1 << 22), "2^22 rows"),
        (dict(temperature=0.0), "temperature"), (dict(temperature=-1.0), "temperature"),
        (dict(temperature=NAN), "temperature"), (dict(temperature=float("inf")), "temperature"),
        (dict(logits_stride=9), "logits_stride"), (dict(dlogits_stride=9), "dlogits_stride"),
        (dict(logits=None), "logits is null"), (dict(logits=A + 1), "logits is null"),
        (dict(dlogits=A + 1), "dlogits is not"), (dict(loss=None), "loss is null"),
        (dict(loss=A + 2), "loss is null"), (dict(weight=A + 2), "weight not"),
        # rows in pieces
        (dict(vocab=50257, logits_stride=50257, dlogits_stride=50257), "workspace"),
        (dict(vocab=50257, logits_stride=50257, dlogits_stride=50257, workspace=A + 8,
              workspace_bytes=1 << 20), "workspace"),
        (dict(vocab=50257, logits_stride=50257, dlogits_stride=50257, workspace=A,
              workspace_bytes=16), "workspace")]


def _refused(call, change, words, base):
    st = call(*{**base, **change}.values())
    assert st in (zr.ZR_ERR_INVALID, zr.ZR_ERR_UNSUPPORTED) and words in zr.zr_last_error()
    assert (st == zr.ZR_ERR_UNSUPPORTED) == ("2^" in words or "1024" in words)


@pytest.mark.parametrize("change,words", BOTH + [
    (dict(ids_type=2), "token type"), (dict(ids=None), "ids is null"), (dict(ids=A + 2), "ids is null"),
    (dict(ids_type=zr.ZR_I64, ids=A + 4), "ids is null"), (dict(teacher_dtype=7), "teacher dtype"),
    (dict(teacher=None), "teacher is null"), (dict(teacher=A + 2), "teacher is null"),
    (dict(ids_stride=3), "ids_stride"), (dict(teacher_stride=3), "teacher_stride"),
    (dict(top=0), "top must"), (dict(top=1025, ids_stride=1025, teacher_stride=1025), "more than 1024"),
])
def test_distill_refusals(change, words):
    _refused(lib.zr_distill_loss, change, words, DISTILL)


@pytest.mark.parametrize("change,words", BOTH + [
    (dict(token_type=2), "token type"), (dict(tokens=None), "tokens is null"),
    (dict(tokens=A + 4), "tokens is null"), (dict(old_logp=None), "old_logp"),
    (dict(advantage=None), "advantage"), (dict(logp=None), "logp"), (dict(ref_logp=None), "kl needs"),
    (dict(ref_logp=A + 2), "element-aligned"), (dict(old_logp=A + 2), "element-aligned"),
    (dict(advantage=A + 1), "element-aligned"), (dict(logp=A + 2), "element-aligned"),
    (dict(clip_low=-0.1), "clip_low"), (dict(clip_low=1.1), "clip_low"), (dict(clip_low=NAN), "clip_low"),
    (dict(clip_high=-0.1), "clip_high"), (dict(clip_high=NAN), "clip_high"),
    (dict(clip_high=float("inf")), "clip_high"), (dict(kl=NAN), "kl must"), (dict(kl=float("inf")), "kl must"),
])
def test_policy_refusals(change, words):
    _refused(lib.zr_policy_loss, change, words, POLICY)


def test_no_rows_need_no_gpu():
    none = dict(logits=None, loss=None, weight=None, dlogits=None, rows=0)
    assert lib.zr_distill_loss(*{**DISTILL, **none, "ids": None, "teacher": None}.values()) == zr.ZR_OK
    none.update(tokens=None, old_logp=None, ref_logp=None, advantage=None, logp=None)
    assert lib.zr_policy_loss(*{**POLICY, **none}.values()) == zr.ZR_OK


def test_workspace():
    n = ctypes.c_int64(7)
    for args in [(-1, 10, 1, 0), (1, 0, 1, 0), (1, 10, 0, 0), (1, 10, 1025, 0), (1, 1 << 30, 1, 0), (1, 10, 1, 2)]:
        assert lib.zr_loss_workspace(*args, ctypes.byref(n)) != zr.ZR_OK and n.value == 0
    assert lib.zr_loss_workspace(1, 10, 1, 0, None) == zr.ZR_ERR_INVALID
    assert zr.zr_loss_workspace(0, 50257, 4, torch.float32) == 0
    assert zr.zr_loss_workspace(200, 128256, 64, torch.bfloat16) == 0
    assert zr.zr_loss_workspace(8192, 128256, 64, torch.bfloat16) == 16
    assert zr.zr_loss_workspace(1, 128256, 64, "bf16") >= 64 * 4
    with pytest.raises(zr.ZrError):
        zr.zr_loss_workspace(1, 10, 1, torch.float16)


def test_host_tensors_are_refused():
    z, f, t = torch.zeros(2, 8), torch.zeros(2), torch.zeros(2, dtype=torch.int64)
    with pytest.raises(zr.ZrError):
        zr.zr_policy_loss(z, t, f, None, f, None, f, f)
    with pytest.raises(zr.ZrError):
        zr.zr_distill_loss(z, t[:, None], z, None, f)
