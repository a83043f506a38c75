"""What the heads and the round decide on the host, on CPU tensors with the device calls replaced
by recorders."""
import pytest
import torch

from speculative_decoding_draft_sample_b200 import binding as bn
from speculative_decoding_draft_sample_b200 import build, heads

V, H, ROWS = 64, 32, 12
BF16 = torch.bfloat16


@pytest.fixture()
def calls(monkeypatch):
    build.build()
    made = []
    for name in ("residual_norm", "linear", "linear_grad", "residual_norm_grad", "token_logprobs"):
        monkeypatch.setattr(bn, name, lambda *a, _n=name, **k: made.append((_n, a, k)))
    return made


def head():
    return heads.LogitHead(torch.ones(H, dtype=BF16), torch.zeros(V, H, dtype=BF16), ROWS)


def bf(*shape):
    return torch.zeros(shape, dtype=BF16)


def test_gradient_needs_the_run_it_belongs_to(calls):
    h = head()
    with pytest.raises(bn.DSparkError, match="after a run of 0"):
        h.gradient(bf(4, V), bf(4, H))
    h.run(bf(4, H), bf(4, V))
    for rows in (3, 5, ROWS):               # rows that the run did not write, or other rows
        with pytest.raises(bn.DSparkError, match="after a run of 4"):
            h.gradient(bf(rows, V), bf(rows, H))
    assert [c[0] for c in calls] == ["residual_norm", "linear"]
    h.gradient(bf(4, V), bf(4, H))
    h.gradient(bf(2, 2, V), bf(2, 2, H))    # again, and in another shape of as many rows
    h.run(bf(ROWS, H), bf(ROWS, V))
    with pytest.raises(bn.DSparkError, match="after a run of 12"):
        h.gradient(bf(4, V), bf(4, H))
    h.gradient(bf(ROWS, V), bf(ROWS, H))
    assert [c[0] for c in calls].count("linear_grad") == 3


def test_a_run_that_failed_leaves_nothing_to_derive(calls, monkeypatch):
    h = head()
    h.run(bf(4, H), bf(4, V))

    def refuse(*a, **k):
        raise bn.DSparkError("refused")

    monkeypatch.setattr(bn, "linear", refuse)
    with pytest.raises(bn.DSparkError, match="refused"):
        h.run(bf(4, H), bf(4, V))
    with pytest.raises(bn.DSparkError, match="after a run of 0"):
        h.gradient(bf(4, V), bf(4, H))


@pytest.mark.parametrize("hidden,logits,delta", [
    ((2, 2 * H), (4, V), None),              # as many values as four rows of H
    ((4, H), (V, 4), None),
    ((4, H), (2, 2 * V), None),
    ((4, H), (4, V), (2, 2 * H)),
    ((4 * H,), (4, V), None),
    ((3, H + 1), (3, V), None),
    ((), (), None),
])
def test_rows_of_another_width_are_refused(calls, hidden, logits, delta):
    with pytest.raises(bn.DSparkError, match="do not fit"):
        head().run(bf(*hidden), bf(*logits), delta=None if delta is None else bf(*delta))
    assert calls == []


@pytest.mark.parametrize("dlogits,dhidden", [((2, 2 * V), (4, H)), ((4, V), (H, 4)), ((V, 4), (4, H)), ((4, V + 1), (4, H)), ((), ())])
def test_gradients_of_another_width_are_refused(calls, dlogits, dhidden):
    h = head()
    h.run(bf(4, H), bf(4, V))
    with pytest.raises(bn.DSparkError, match="do not fit"):
        h.gradient(bf(*dlogits), bf(*dhidden))
    assert len(calls) == 2


def test_rows_may_be_shaped_otherwise_on_either_side(calls):
    h = head()
    h.run(bf(2, 2, H), bf(4, V), delta=bf(4, 1, H))
    h.run(bf(4, H), bf(2, 2, V))
    h.gradient(bf(2, 2, V), bf(4, H))
    assert [c[0] for c in calls] == ["residual_norm", "linear"] * 2 + ["linear_grad", "residual_norm_grad"]


def test_scores_keep_their_buffers_between_counts_of_alternatives(calls):
    """A graph may still write the buffers of an earlier call with another n_top."""
    from speculative_decoding_draft_sample_b200.spec_round import SpecRound
    rnd = SpecRound(2, 3, V, 64, device="cpu")
    rnd.verified = bf(2, 4, V)
    five, none = rnd.score(None, n_top=5), rnd.score(None)
    places = [t.data_ptr() for t in (five.logp, five.top_idx, five.ws)]
    del five
    taken = {none.logp.data_ptr(), none.ws.data_ptr()} | {torch.zeros_like(none.ws).data_ptr() for _ in range(8)}
    again = rnd.score(None, n_top=5)
    assert [t.data_ptr() for t in (again.logp, again.top_idx, again.ws)] == places
    assert not taken & set(places)
    assert rnd.scores is again and rnd.score(None) is none
    assert [c[1][3].data_ptr() for c in calls] == [again.logp.data_ptr(), none.logp.data_ptr()] * 2
