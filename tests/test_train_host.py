"""The operators' C ABI without a GPU: every declared entry point is there, and bad arguments are refused on the host,
before anything reaches a device, with the documented status."""
import ctypes
import math

import pytest

import clip_tensor_adamw_gb300 as mica
from clip_tensor_adamw_gb300 import train

OK, NULL, COUNT, DTYPE, HYPER = 0, 1, 2, 3, 4
F32, F16, BF16X2, BF16 = 0, 1, 2, 4


def logits(**kw):
    d = dict(logits=0x1000, targets=0x2000, rows=4, vocab=100, ld=100, temperature=1.0, dtype=F32, target_bytes=8)
    d.update(kw)
    return train._Logits(*(d[k] for k, _ in train._Logits._fields_))


def packed(**kw):
    d = dict(codes=0x1000, steps=0x2000, rows=4, cols=100, ld=128, ld_s=4, dtype=BF16, reserved=0)
    d.update(kw)
    return train._Packed(*(d[k] for k, _ in train._Packed._fields_))


def pref(**kw):
    d = dict(beta=0.1, label_smoothing=0.0, grad_scale=1.0, kind=0, flags=0)
    d.update(kw)
    return train._PreferenceHP(*(d[k] for k, _ in train._PreferenceHP._fields_))


def policy(**kw):
    d = dict(clip_low=0.2, clip_high=0.2, kl_coef=0.0, denom=1.0, grad_scale=1.0)
    d.update(kw)
    return train._PolicyHP(*(d[k] for k, _ in train._PolicyHP._fields_))


BAD_LOGITS = [(dict(dtype=BF16X2), DTYPE), (dict(dtype=7), DTYPE), (dict(target_bytes=2), DTYPE),
              (dict(temperature=0.0), HYPER), (dict(temperature=math.nan), HYPER), (dict(temperature=math.inf), HYPER),
              (dict(temperature=1e-31), HYPER), (dict(temperature=1e31), HYPER), (dict(rows=-1), COUNT),
              (dict(rows=(1 << 30) + 1), COUNT), (dict(vocab=0), COUNT), (dict(vocab=(1 << 24) + 1), COUNT),
              (dict(ld=-1), COUNT)]


@pytest.mark.parametrize("bad,want", BAD_LOGITS)
def test_logits_are_checked_by_every_call(bad, want):
    L = train._train()
    z = logits(**bad)
    assert L.mica_token_logps(z, 0x3000, None, None) == want
    assert L.mica_token_logps_grad(z, 0x3000, 0x4000, 1 << 25, None) == want
    assert L.mica_preference_loss(z, 0x3000, 1, None, pref(), 0x4000, None, 0x5000, None, 0, 0x6000, 1 << 20, None) == want
    assert L.mica_policy_loss(z, 0x3000, 0x4000, None, None, policy(), 0x5000, 0x6000, None, 0, None) == want


def test_no_rows_need_no_device():
    L = train._train()
    assert L.mica_token_logps(logits(rows=0), None, None, None) == OK
    assert L.mica_token_logps_grad(logits(rows=0), None, None, 100, None) == OK
    assert L.mica_act_pack(None, 100, packed(rows=0), 0, 0, None, 0, None) == OK
    assert L.mica_act_unpack(packed(rows=0), None, 100, None) == OK
    assert L.mica_act_grad(packed(cols=0), 1, 0, None, 0, F32, None, 0, None) == OK
    assert L.mica_packed_wgrad(packed(), None, 0, BF16, 0, None, 0, None, 0, F32, None, 0, None) == OK


def test_losses_host_validation():
    L = train._train()
    assert L.mica_token_logps(None, 0x3000, None, None) == NULL
    assert L.mica_token_logps_grad(logits(), 0x3000, 0x4000, 99, None) == COUNT

    def p(hp=None, pairs=1, work=0x6000, size=1 << 20, ld=100, **kw):
        return L.mica_preference_loss(logits(**kw), 0x3000, pairs, None, hp, 0x4000, None, 0x5000, 0x7000, ld, work, size, None)

    assert p(None) == NULL
    assert p(pref(), pairs=-1) == COUNT and p(pref(), pairs=(1 << 24) + 1) == COUNT and p(pref(), ld=99) == COUNT
    assert p(pref(), work=None) == NULL
    assert p(pref(), size=L.mica_preference_workspace(4, 1) - 1) == COUNT
    for bad in (dict(beta=0.0), dict(beta=-1.0), dict(beta=math.inf), dict(label_smoothing=1.0), dict(label_smoothing=-0.1),
                dict(label_smoothing=math.nan), dict(kind=1, label_smoothing=0.1), dict(kind=3), dict(kind=-1),
                dict(grad_scale=math.nan), dict(flags=2)):
        assert p(pref(**bad)) == HYPER, bad

    def q(hp, ld=100):
        return L.mica_policy_loss(logits(), 0x3000, 0x4000, None, None, hp, 0x5000, 0x6000, 0x7000, ld, None)

    assert q(None) == NULL and q(policy(), ld=99) == COUNT
    for bad in (dict(clip_low=-0.1), dict(clip_low=1.1), dict(clip_low=math.nan), dict(clip_high=-0.1),
                dict(clip_high=math.nan), dict(kl_coef=-1.0), dict(kl_coef=math.inf), dict(denom=0.0), dict(denom=-1.0),
                dict(denom=math.inf), dict(grad_scale=math.inf)):
        assert q(policy(**bad)) == HYPER, bad


def test_workspace_sizes():
    L = train._train()
    assert L.mica_preference_workspace(0, 0) == 0
    assert L.mica_preference_workspace(-1, 1) == 0 and L.mica_preference_workspace(1, -1) == 0
    assert L.mica_preference_workspace(1000, 4) >= 1000 * 16 + 4 * 16


def test_checkpoints_host_validation():
    L = train._train()
    for bad, want in ((dict(dtype=2), DTYPE), (dict(rows=-1), COUNT), (dict(cols=-1), COUNT), (dict(cols=(1 << 24) + 1), COUNT),
                      (dict(ld=96), COUNT), (dict(ld=120), COUNT), (dict(ld_s=3), COUNT), (dict(ld_s=5), COUNT)):
        p = packed(**bad)
        assert L.mica_act_pack(0x3000, 100, p, 0, 0, None, 0, None) == want, bad
        assert L.mica_act_unpack(p, 0x3000, 200, None) == want, bad
        assert L.mica_act_grad(p, 1, 0, 0x3000, 100, F32, 0x4000, 200, None) == want, bad
        assert L.mica_packed_wgrad(p, 0x3000, 8, BF16, 8, None, 0, 0x4000, 8, F32, None, 0, None) == want, bad
    assert L.mica_act_pack(0x3000, 100, None, 0, 0, None, 0, None) == NULL
    p = packed()
    assert L.mica_act_pack(0x3000, 100, p, 5, 0, 0x4000, 100, None) == HYPER
    assert L.mica_act_pack(0x3000, 100, p, -1, 0, 0x4000, 100, None) == HYPER
    assert L.mica_act_pack(0x3000, 100, p, 0, 1, None, 0, None) == HYPER       # gated without a function
    assert L.mica_act_pack(0x3000, 100, p, 0, 0, 0x4000, 100, None) == HYPER   # y without a function
    assert L.mica_act_pack(0x3000, 100, p, 3, 1, 0x4000, 50, None) == COUNT    # 100 is not twice a multiple of 32
    assert L.mica_act_pack(0x3000, 100, p, 3, 0, 0x4000, 99, None) == COUNT
    assert L.mica_act_unpack(p, 0x3000, 99, None) == COUNT
    assert L.mica_act_grad(p, 0, 0, 0x3000, 100, F32, 0x4000, 100, None) == HYPER
    assert L.mica_act_grad(p, 1, 0, 0x3000, 100, 3, 0x4000, 100, None) == DTYPE
    assert L.mica_act_grad(p, 1, 0, 0x3000, 100, F32, 0x4000, 99, None) == COUNT


def test_wgrad_host_validation():
    L = train._train()

    def w(p=None, dy=BF16, n=8, ld_dy=8, ld_dw=8, dw=F32):
        return L.mica_packed_wgrad(p or packed(), 0x3000, ld_dy, dy, n, None, 0, 0x4000, ld_dw, dw, None, 0, None)

    assert w(dy=F32) == DTYPE and w(dw=2) == DTYPE
    assert w(dy=F16) == DTYPE                       # a float16 dy needs a float16 checkpoint
    assert w(n=-1) == COUNT and w(ld_dy=-1) == COUNT and w(ld_dw=7) == COUNT


def test_python_checks_need_no_device():
    import torch
    z, y = torch.zeros(4, 10), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(TypeError):
        mica.mica_token_logps(z.double(), y)
    with pytest.raises(TypeError):
        mica.mica_token_logps(z, y.float())
    with pytest.raises(ValueError):
        mica.mica_token_logps(z, y[:2])
    with pytest.raises(ValueError):
        mica.mica_token_logps(z[0], y[:1])
    with pytest.raises(ValueError):
        mica.mica_preference_loss(z, y, torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError):
        mica.mica_preference_loss(z, y, torch.zeros(3, dtype=torch.int32), kind="x")
    with pytest.raises(TypeError):
        mica.mica_policy_loss(z, y, torch.zeros(4).double(), torch.zeros(4), denom=1.0)
    with pytest.raises(TypeError):
        mica.PackedActivation(torch.zeros(4, 32), torch.zeros(4, 4, dtype=torch.uint8), 32, torch.float32)
    with pytest.raises(ValueError):
        mica.PackedActivation(torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4, 4, dtype=torch.uint8), 33, torch.float32)
    p = mica.PackedActivation.empty(4, 33, torch.float16, "cpu")
    assert p.codes.shape == (4, 64) and p.steps.shape == (4, 4) and p.shape == (4, 33)
    with pytest.raises(ValueError):
        mica.mica_act_grad(p, torch.zeros(4, 32), "silu")


def test_spans_that_would_wrap_are_refused():
    """(rows - 1) * ld + columns elements in bytes may pass 64 bits with each factor in its range; such a matrix is refused
    before anything else looks at it, on a machine without a GPU too."""
    L = train._train()
    for rows, ld in (((1 << 24) + 1, 1 << 40), (1 << 30, 1 << 40), ((1 << 22) + 1, 1 << 40), (1 << 24, 1 << 40)):
        z = logits(rows=rows, ld=ld)
        assert L.mica_token_logps(z, 0x3000, None, None) == COUNT
        assert L.mica_token_logps_grad(z, 0x3000, 0x4000, 100, None) == COUNT
        assert L.mica_preference_loss(z, 0x3000, 1, None, pref(), 0x4000, None, 0x5000, None, 0, 0x6000, 1 << 40, None) == COUNT
        assert L.mica_policy_loss(z, 0x3000, 0x4000, None, None, policy(), 0x5000, 0x6000, None, 0, None) == COUNT
        z = logits(rows=rows)
        assert L.mica_token_logps_grad(z, 0x3000, 0x4000, ld, None) == COUNT
        assert L.mica_preference_loss(z, 0x3000, 1, None, pref(), 0x4000, None, 0x5000, 0x7000, ld, 0x6000, 1 << 40,
                                      None) == COUNT
        assert L.mica_policy_loss(z, 0x3000, 0x4000, None, None, policy(), 0x5000, 0x6000, 0x7000, ld, None) == COUNT
        for wide in (dict(ld=ld), dict(ld_s=ld)):
            p = packed(rows=rows, **wide)
            assert L.mica_act_pack(0x3000, 100, p, 0, 0, None, 0, None) == COUNT
            assert L.mica_act_unpack(p, 0x3000, 100, None) == COUNT
            assert L.mica_act_grad(p, 1, 0, 0x3000, 100, F32, 0x4000, 100, None) == COUNT
            assert L.mica_packed_wgrad(p, 0x3000, 8, BF16, 8, None, 0, 0x4000, 8, F32, None, 0, None) == COUNT
        p = packed(rows=rows)
        assert L.mica_act_pack(0x3000, ld, p, 0, 0, None, 0, None) == COUNT
        assert L.mica_act_pack(0x3000, 100, p, 3, 0, 0x4000, ld, None) == COUNT
        assert L.mica_act_unpack(p, 0x3000, ld, None) == COUNT
        assert L.mica_act_grad(p, 1, 0, 0x3000, ld, F32, 0x4000, 100, None) == COUNT
        assert L.mica_act_grad(p, 1, 0, 0x3000, 100, F32, 0x4000, ld, None) == COUNT
        assert L.mica_packed_wgrad(p, 0x3000, ld, BF16, 8, None, 0, 0x4000, 8, F32, None, 0, None) == COUNT
    p = packed(cols=1 << 24, ld=1 << 24, ld_s=1 << 20)
    for add, ld_add, ld_dw in ((None, 0, 1 << 40), (0x5000, 1 << 40, 8)):
        assert L.mica_packed_wgrad(p, 0x3000, 8, BF16, 8, add, ld_add, 0x4000, ld_dw, F32, None, 0, None) == COUNT
    assert L.mica_packed_wgrad(p, 0x3000, 1 << 24, BF16, 1 << 24, None, 0, 0x4000, 1 << 24, F32, None, 0, None) == COUNT
    assert L.mica_packed_wgrad_workspace(p, 0x3000, 1 << 24, 1 << 24) == 0
    # one row may have any stride: it spans its columns
    assert L.mica_act_unpack(packed(rows=1, ld=1 << 40), None, 1 << 40, None) not in (OK, COUNT)


def test_a_gradient_takes_no_more_memory_than_its_rows():
    """The logits of the last tokens of a batch are far apart; their gradient is not, and lies as they do within 128 bytes."""
    import torch
    batch = torch.zeros(3, 7, 1009, dtype=torch.bfloat16)
    for z in (batch[:, -1], batch[:, 3, :1000], torch.zeros(5, 1024)[:, :1009], torch.zeros(5, 1009),
              torch.zeros(4, 1, 130)[:, 0], torch.zeros(1, 64).expand(6, 64)):
        ld = train._matrix(z, "logits")
        d = train._dlogits(None, z, ld)
        assert d.shape == z.shape and d.dtype == z.dtype
        line = 128 // z.element_size()
        assert d.untyped_storage().nbytes() <= z.shape[0] * (z.shape[1] + line - 1) * z.element_size()
        if ld > z.shape[1]:
            assert (train._matrix(d, "dlogits") - ld) % line == 0
