"""Which step number the optimizer hands to the library for which parameter (no GPU: the library's step is
replaced by a recorder)."""
import io
import random

import pytest
import torch

from kimi_delta_attention_gb300 import adamw
from kimi_delta_attention_gb300.adamw import AdamW


@pytest.fixture
def calls(monkeypatch):
    """Every call's (params, step number, learning rate)."""
    got = []

    def record(params, grads, exp_avgs, exp_avg_sqs, step, lr, **kw):
        got.append((list(params), int(step), float(lr)))

    monkeypatch.setattr(adamw, "kda_adamw_step", record)
    return got


def parameters(n):
    return [torch.nn.Parameter(torch.zeros(3)) for _ in range(n)]


def take(opt, params, which):
    for i, p in enumerate(params):
        p.grad = torch.ones_like(p) if i in which else None
    opt.step()


def counts(calls, params):
    """{parameter's number: the step numbers it was given}; the list is emptied."""
    out = {i: [] for i in range(len(params))}
    for some, step, _ in calls:
        for p in some:
            out[next(i for i, q in enumerate(params) if q is p)].append(step)
    calls.clear()
    return out


@pytest.mark.parametrize("capturable", [False, True])
def test_a_late_parameter_counts_from_one(calls, capturable):
    params = parameters(3)
    opt = AdamW(params, capturable=capturable)
    for k in range(6):
        take(opt, params, {0, 2} if k < 4 else {0, 1, 2})
    assert counts(calls, params) == {0: [1, 2, 3, 4, 5, 6], 1: [1, 2], 2: [1, 2, 3, 4, 5, 6]}


@pytest.mark.parametrize("capturable", [False, True])
@pytest.mark.parametrize("seed", range(5))
def test_each_parameter_counts_its_own_steps(calls, capturable, seed):
    rng = random.Random(seed)
    params = parameters(7)
    opt = AdamW([dict(params=params[:4]), dict(params=params[4:])], capturable=capturable)
    want = {i: [] for i in range(7)}
    for _ in range(12):
        which = {i for i in range(7) if rng.random() < 0.7}
        for i in which:
            want[i].append(len(want[i]) + 1)
        take(opt, params, which)
    assert counts(calls, params) == want


def test_parameters_that_step_together_share_a_call(calls):
    """Also after one has missed a step: those that go on keep the group's word, which a captured step reads."""
    params = parameters(5)
    opt = AdamW(params, capturable=True)
    take(opt, params, range(5))
    word = opt.param_groups[0]["step_device"]
    take(opt, params, {0, 1, 2})
    take(opt, params, range(5))
    assert [len(some) for some, _, _ in calls] == [5, 3, 3, 2]
    assert word is opt.param_groups[0]["step_device"] and word.item() == 3
    assert [opt.state[p]["step_device"] is word for p in params] == [True] * 3 + [False] * 2


@pytest.mark.parametrize("capturable", [False, True])
def test_a_group_on_two_devices(monkeypatch, capturable):
    """Each device's parameters with words of that device, each counted once a step."""
    got = []
    monkeypatch.setattr(adamw, "kda_adamw_step", lambda params, g, m, v, step, **kw: got.append((params[0].device, step, kw)))
    params = [torch.nn.Parameter(torch.zeros(3, device=d)) for d in ("cpu", "meta", "cpu")]
    opt = AdamW(params, lr=0.5, capturable=capturable)
    for _ in range(3):
        for p in params:
            p.grad = torch.ones_like(p)
        opt.step(grad_scale=torch.ones(1), skip=torch.zeros(1))
    assert [d.type for d, _, _ in got] == ["cpu", "meta"] * 3
    for device, step, kw in got:
        words = [kw["grad_scale"], kw["skip"]] + ([step, kw["lr"]] if capturable else [])
        assert all(t.device == device and t.numel() == 1 for t in words)
    if capturable:
        assert opt.state[params[0]]["step_device"].item() == 3 and opt.state[params[0]]["step_device"] is opt.state[params[2]]["step_device"]
        assert got[1][1] is got[3][1] is got[5][1]
    assert [opt.state[p]["step"] for p in params] == [3, 3, 3]


def through_a_file(opt):
    file = io.BytesIO()
    torch.save(opt.state_dict(), file)
    file.seek(0)
    return torch.load(file, map_location="cpu", weights_only=False)


@pytest.mark.parametrize("capturable", [False, True])
def test_counts_go_on_after_a_file(calls, capturable):
    params, twin = parameters(5), parameters(5)
    opt = AdamW([dict(params=params[:4]), dict(params=params[4:], lr=0.25)], lr=0.125, capturable=capturable)
    for which in (range(3), {0, 1, 4}, range(3)):
        take(opt, params, which)
    other = AdamW([dict(params=twin[:4]), dict(params=twin[4:])], capturable=capturable)
    other.load_state_dict(through_a_file(opt))
    calls.clear()
    take(other, twin, range(5))
    assert [(len(some), step, lr) for some, step, lr in calls] == [(2, 4, 0.125), (1, 3, 0.125), (1, 1, 0.125), (1, 2, 0.25)]
    if capturable:                              # the group's word is again the one of those that stepped at every step
        assert other.param_groups[0]["step_device"] is other.state[twin[0]]["step_device"]


def test_counts_of_a_file_without_words_by_parameter(calls):
    """A capturable group saved with its one word (which replays advance, and host counts do not follow)."""
    params, twin = parameters(3), parameters(3)
    opt = AdamW(params, capturable=True)
    take(opt, params, {0, 1})
    old = through_a_file(opt)
    old["param_groups"][0]["step_device"].fill_(9)
    for state in old["state"].values():
        del state["step_device"]
    other = AdamW(twin, capturable=True)
    other.load_state_dict(old)
    calls.clear()
    take(other, twin, range(3))
    assert counts(calls, twin) == {0: [10], 1: [10], 2: [1]}


@pytest.mark.parametrize("capturable", [False, True])
def test_a_refused_call_counts_nothing(calls, monkeypatch, capturable):
    params = parameters(2)
    opt = AdamW(params, capturable=capturable)
    take(opt, params, {0, 1})
    with monkeypatch.context() as m:
        m.setattr(adamw, "kda_adamw_step", refuse)
        with pytest.raises(adamw.KdaError):
            take(opt, params, {0, 1})
    calls.clear()
    take(opt, params, {0, 1})
    assert counts(calls, params) == {0: [2], 1: [2]} and opt.state[params[0]]["step"] == 2


def refuse(*a, **kw):
    raise adamw.KdaError(1, "not contiguous")


def test_what_a_capture_would_make_anew_is_refused(calls, monkeypatch):
    params = parameters(3)
    opt = AdamW(params, capturable=True)
    with monkeypatch.context() as m:
        m.setattr(adamw, "_capturing", lambda: True)
        with pytest.raises(adamw.KdaError, match="state"):
            take(opt, params, {0, 1})
    take(opt, params, {0, 1})
    calls.clear()
    with monkeypatch.context() as m:
        m.setattr(adamw, "_capturing", lambda: True)
        with pytest.raises(adamw.KdaError, match="state"):              # one joins
            take(opt, params, {0, 1, 2})
        with pytest.raises(adamw.KdaError, match="apart"):              # one stays behind
            take(opt, params, {0})
        take(opt, params, {0, 1})
        opt.param_groups[0]["lr"] = 0.5
        with pytest.raises(adamw.KdaError, match="learning rate"):
            take(opt, params, {0, 1})
        plain = AdamW(params)
        with pytest.raises(adamw.KdaError, match="capturable=True"):
            take(plain, params, {0})
    opt.param_groups[0]["lr"] = 0.5
    take(opt, params, {0, 1, 2})
    assert [step for _, step, _ in calls] == [2, 3, 1]


def test_words_of_another_device_are_not_copied_under_capture(calls, monkeypatch):
    params = parameters(1)
    opt = AdamW(params, capturable=True)
    take(opt, params, {0})
    calls.clear()
    word = opt.state[params[0]]["step_device"]
    opt.param_groups[0]["lr"] = opt.param_groups[0]["lr"].to("meta")
    monkeypatch.setattr(adamw, "_capturing", lambda: True)
    with pytest.raises(adamw.KdaError, match="word on cpu"):
        take(opt, params, {0})
    assert not calls and word.item() == 1


def test_counts_when_a_group_changes_its_mode(calls):
    """Replays advance the words and not the host's counts; a group that is no longer capturable goes on from the
    words, and one that becomes capturable from the counts."""
    params = parameters(3)
    opt = AdamW(params, capturable=True)
    take(opt, params, {0, 1})
    opt.state[params[0]]["step_device"].add_(5)                     # (as replays do)
    group = opt.param_groups[0]
    group["capturable"] = False
    take(opt, params, {0, 2})
    group["capturable"] = True
    calls.clear()
    take(opt, params, {0, 1, 2})
    assert counts(calls, params) == {0: [8], 1: [7], 2: [2]}
