"""Routing rules without a GPU: refusals of the C calls and of the binding, and the reference
itself against hand-made cases.  Pointers are fake and never dereferenced."""
import ctypes

import numpy as np
import pytest

import quantized_sparse_moe_amd as q
import rule_ref
from test_abi_cpu import FAKE, desc


def rule(**kw):
    r = q.moe_router_rule(q.MOE_SCORE_SIGMOID, 1, 8, 4, q.MOE_GROUP_TOP2, 2.5, FAKE)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def select(r, logits=FAKE, dtype=q.MOE_F32, T=4, E=256, ld=256, k=8, idx=FAKE, w=FAKE):
    return q.lib().moe_select(None if r is None else ctypes.byref(r), logits, dtype, T, E, ld, k, idx, w, None)


@pytest.mark.parametrize("field,value,status", [
    ("score", 2, q.MOE_ERR_INVALID), ("score", -1, q.MOE_ERR_INVALID), ("renorm", 2, q.MOE_ERR_INVALID),
    ("group_score", 2, q.MOE_ERR_INVALID), ("scale", float("nan"), q.MOE_ERR_INVALID),
    ("scale", float("inf"), q.MOE_ERR_INVALID), ("select_bias", FAKE + 2, q.MOE_ERR_INVALID),
    ("n_groups", 0, q.MOE_ERR_INVALID), ("group_top_k", 0, q.MOE_ERR_INVALID), ("group_top_k", 9, q.MOE_ERR_INVALID),
    ("n_groups", 7, q.MOE_ERR_UNSUPPORTED), ("n_groups", 128, q.MOE_ERR_UNSUPPORTED)])
def test_rule_fields_are_checked(field, value, status):
    r = rule(**{field: value})
    assert select(r) == status
    d = desc()
    assert q.lib().moe_route_rule(ctypes.byref(d), ctypes.byref(r), FAKE, 4, FAKE, FAKE, FAKE, 1 << 40, None) == status
    assert q.lib().moe_layer_forward_rule(ctypes.byref(d), ctypes.byref(r), FAKE, 4, FAKE, q.MOE_F32, None, None, FAKE,
                                          1 << 40, None) == status


def test_groups_must_hold_the_selection():
    assert select(rule(n_groups=64, group_top_k=2), k=9) == q.MOE_ERR_UNSUPPORTED       # 8 experts stay
    assert select(rule(n_groups=64, group_top_k=2), k=8, T=0) == q.MOE_OK


def test_select_arguments():
    assert select(None) == q.MOE_ERR_INVALID
    assert select(rule(), logits=None) == q.MOE_ERR_INVALID
    assert select(rule(), logits=FAKE + 2) == q.MOE_ERR_INVALID                         # fp32 needs 4 bytes
    assert select(rule(), dtype=q.MOE_E8M0) == q.MOE_ERR_INVALID
    assert select(rule(), ld=255) == q.MOE_ERR_INVALID
    assert select(rule(), idx=None) == q.MOE_ERR_INVALID
    assert select(rule(), w=FAKE + 2) == q.MOE_ERR_INVALID
    assert select(rule(), T=-1) == q.MOE_ERR_INVALID
    assert select(rule(), T=(1 << 20) + 1) == q.MOE_ERR_UNSUPPORTED
    assert select(rule(), E=0) == q.MOE_ERR_UNSUPPORTED
    assert select(rule(), E=264, ld=264) == q.MOE_ERR_UNSUPPORTED
    assert select(rule(), k=0) == q.MOE_ERR_UNSUPPORTED
    assert select(rule(), k=17) == q.MOE_ERR_UNSUPPORTED
    assert select(rule(n_groups=1, group_top_k=1), E=4, k=5) == q.MOE_ERR_UNSUPPORTED
    assert select(rule(), logits=None, T=0) == q.MOE_OK
    far = dict(idx=FAKE + (1 << 32), w=FAKE + (2 << 32))
    for kw in (dict(far, idx=FAKE + 4092), dict(far, w=FAKE), dict(far, w=far["idx"] + 124), dict(far, logits=far["w"] + 64)):
        assert select(rule(), **kw) == q.MOE_ERR_INVALID, kw        # (T = 4: 4096 bytes of logits, 128 of results)


def test_select_results_over_the_bias_are_refused():
    far = dict(idx=FAKE + (1 << 32), w=FAKE + (2 << 32), logits=FAKE + (3 << 32))
    for kw in (dict(idx=FAKE), dict(w=FAKE + 1020), dict(w=FAKE - 124)):     # (256 values of bias, 128 bytes of results)
        assert select(rule(), **dict(far, **kw)) == q.MOE_ERR_INVALID, kw


def test_layer_calls_need_a_rule_and_keep_their_checks():
    L, d, r = q.lib(), desc(), rule()
    fwd = lambda d, r, x=FAKE, T=4, yt=q.MOE_F32, ws=FAKE, n=1 << 40: L.moe_layer_forward_rule(
        ctypes.byref(d), r, x, T, FAKE, yt, None, None, ws, n, None)
    assert fwd(d, None) == q.MOE_ERR_INVALID
    assert fwd(d, ctypes.byref(r), x=None) == q.MOE_ERR_INVALID
    assert fwd(d, ctypes.byref(r), yt=q.MOE_F16) == q.MOE_ERR_INVALID
    assert fwd(d, ctypes.byref(r), ws=None) == q.MOE_ERR_WORKSPACE
    assert fwd(d, ctypes.byref(r), n=1 << 20) == q.MOE_ERR_WORKSPACE
    assert fwd(desc(top_k=0), ctypes.byref(r)) == q.MOE_ERR_UNSUPPORTED
    assert fwd(d, ctypes.byref(r), x=None, T=0) == q.MOE_OK
    assert L.moe_route_rule(ctypes.byref(d), None, FAKE, 4, FAKE, FAKE, FAKE, 1 << 40, None) == q.MOE_ERR_INVALID
    assert L.moe_route_rule(ctypes.byref(d), ctypes.byref(r), FAKE, 4, None, FAKE, FAKE, 1 << 40, None) == q.MOE_ERR_INVALID


def test_rule_object_checks_its_arguments():
    import torch
    for bad in (dict(score="relu"), dict(group_score="sum"), dict(select_bias=torch.zeros(4, dtype=torch.bfloat16)),
                dict(select_bias=torch.zeros(2, 2)), dict(select_bias=torch.zeros(8)[::2])):
        with pytest.raises(q.QsmoeError):
            q.RouterRule(**bad)
    r = q.RouterRule(score="sigmoid", renorm=False, n_groups=4, group_top_k=2, group_score="top2", scale=0.5)
    d = r.desc
    assert (d.score, d.renorm, d.n_groups, d.group_top_k, d.group_score, d.scale) == (1, 0, 4, 2, 1, 0.5)
    with pytest.raises(q.QsmoeError):
        q.moe_select(torch.zeros(2, 8), 2, q.RouterRule(select_bias=torch.zeros(9)))
    with pytest.raises(q.QsmoeError):                       # host tensors
        q.moe_select(torch.zeros(2, 8), 2, q.RouterRule())
    with pytest.raises(q.QsmoeError):
        q.moe_select(torch.zeros(2, 8), 2, q.RouterRule(), topk_idx=torch.zeros(2, 3, dtype=torch.int32))
    with pytest.raises(q.QsmoeError):
        q.moe_select(torch.zeros(2, 8), 2, q.RouterRule(), topk_w=torch.zeros(2, 2, dtype=torch.float64))


def test_tensors_whose_addresses_are_held_cannot_be_replaced():
    """A call after such an assignment would read the old tensor, which may be gone; writes into the tensors go
    through."""
    import torch
    bf = torch.bfloat16
    rule = q.RouterRule(score="sigmoid", select_bias=torch.zeros(8))
    norm = q.Norm(weight=torch.ones(8), bias=torch.zeros(8))
    ad = q.LoraAdapters(torch.zeros(2, 8, 16, dtype=bf), torch.zeros(2, 24, 8, dtype=bf), scales=torch.ones(2))
    for o, name in ((rule, "select_bias"), (norm, "weight"), (norm, "bias"), (ad, "a"), (ad, "b"), (ad, "scales"), (ad, "ranks"),
                    (ad, "N")):
        old = getattr(o, name)
        with pytest.raises(q.QsmoeError):
            setattr(o, name, torch.ones(8))
        assert getattr(o, name) is old
    rule.select_bias += 1
    norm.weight[:] = 2.0
    assert rule.desc.select_bias == rule.select_bias.data_ptr() and (rule.select_bias == 1).all()


def test_reference_by_hand():
    l = np.log(np.array([[1.0, 2.0, 4.0, 1.0, 3.0, 5.0, 0.0, 0.0]]) + 0.0, where=np.array([[1] * 6 + [0] * 2], bool),
               out=np.full((1, 8), -np.inf))
    i, w, gap = rule_ref.select(l, 2, score="softmax", renorm=True)
    assert i.tolist() == [[2, 5]] and np.allclose(w, [[4 / 9, 5 / 9]])
    i, w, _ = rule_ref.select(l, 2, score="softmax", renorm=False, scale=2.0)
    assert np.allclose(w, [[8 / 16, 10 / 16]])
    # groups of two: {1, 2} {4, 1} {3, 5} {-}: by their best 3, 2; by their two best the same
    i, w, _ = rule_ref.select(l, 2, n_groups=4, group_top_k=1, group_score="top2")
    assert i.tolist() == [[4, 5]]
    # nothing else is left: masked experts, lowest first, weight 0
    i, w, _ = rule_ref.select(np.full((1, 4), -np.inf), 2)
    assert i.tolist() == [[0, 1]] and not w.any()
    # ties to the lower expert, a bias changes the choice and not the weight
    i, w, gap = rule_ref.select(np.zeros((1, 4)), 2, score="sigmoid", renorm=False)
    assert i.tolist() == [[0, 1]] and np.allclose(w, 0.5) and gap[0] == 0
    i, w, _ = rule_ref.select(np.zeros((1, 4)), 2, score="sigmoid", renorm=False, select_bias=np.array([0, 0, 1, 2.0]))
    assert i.tolist() == [[2, 3]] and np.allclose(w, 0.5)
