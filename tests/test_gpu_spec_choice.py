"""What the batched model's calls take as a sequence's choice around tree steps
and acceptances."""
import numpy as np
import pytest

from transformer_decode_token_gb300 import binding, synth

pytestmark = pytest.mark.gpu


def refused(call):
    with pytest.raises(binding.GPT2Error) as e:
        call()
    return e.value.name


@pytest.mark.parametrize("kv", ["f32", "int8"])
def test_a_tree_step_makes_no_choice(kv):
    """On a new model a tree step leaves logits but nothing to go on from; the
    acceptance does."""
    cfg = synth.TINY
    m = binding.BatchModel(cfg, binding.upload_weights(synth.make_weights(cfg, 0)), 8, kv=kv)
    try:
        assert refused(lambda: m.argmax(2)) == "NOT_READY"
        m.decode_tree([([5, 9], [-1, 0]), ([7], [-1])])
        assert np.isfinite(m.logits(3)).all()
        assert refused(lambda: m.argmax(2)) == "NOT_READY"
        assert refused(lambda: m.decode_greedy(1)) == "NOT_READY"
        got = m.accept_tree()
        assert m.argmax(2) == [g[-1] for g in got]
        m.decode_greedy(2)
        m.sync()
    finally:
        m.close()


def test_no_choice_is_not_an_earlier_one():
    """A sequence whose acceptance ends without a choice has none: its earlier
    choice is not returned, and greedy steps refuse until it has been given a
    token, then go on as those of a model that decoded the same tokens."""
    cfg = synth.TINY
    w = dict(synth.make_weights(cfg, 0))
    w["wpe"] = np.array(w["wpe"])
    w["wpe"][9] = np.nan
    m = binding.BatchModel(cfg, binding.upload_weights(w), 8)
    ref = binding.BatchModel(cfg, binding.upload_weights(synth.make_weights(cfg, 0)), 8)
    try:
        prompts = [[1, 2, 3], [4, 5, 6, 7, 8, 9, 10, 11, 12]]     # the second's next position is 9
        m.prefill(prompts)
        ref.prefill(prompts[:1])
        first = m.argmax(2)
        m.decode_tree([([first[0], 5], [-1, 0]), ([first[1], 6], [-1, 0])])
        ref.decode_tree([([first[0], 5], [-1, 0])])
        want = ref.accept_tree()
        assert refused(m.accept_tree) == "DEVICE_STATE"
        assert m.argmax(2) == [want[0][-1], -1]
        assert refused(lambda: m.decode_greedy(1)) == "NOT_READY"
        assert refused(lambda: m.decode_greedy(0)) == "NOT_READY"
        # a new prompt for the second (the first's again, with what it gained)
        ids = prompts[0] + [first[0]] + want[0][:-1]
        m.prefill([ids, prompts[0]])
        ref.prefill([ids, prompts[0]])
        m.decode_greedy(3)
        ref.decode_greedy(3)
        assert m.argmax(2) == ref.argmax(2)
        # or a token
        m.prefill(prompts)
        m.decode_tree([None, (m.argmax(2)[1:], [-1])])
        assert refused(m.accept_tree) == "DEVICE_STATE"
        m.decode([0, 3], [-1, 0])
        m.decode_greedy(1)
        m.sync()
    finally:
        m.close()
        ref.close()


@pytest.mark.parametrize("own_stream", [False, True])
def test_acceptance_waits_for_its_tensors(own_stream):
    """Probabilities and random numbers that another stream is still making when
    accept_tree is called there: the tokens are those of the finished tensors.
    Tensors elsewhere than on the model's device are refused."""
    import torch
    cfg = synth.TINY
    V = cfg.vocab_size
    rng = np.random.default_rng(4)
    ours = torch.cuda.Stream() if own_stream else None
    m = binding.BatchModel(cfg, binding.upload_weights(synth.make_weights(cfg, 0)), 16, stream=ours)
    try:
        torch.cuda.synchronize()
        tree = [([5, 9, 11, 2], [-1, 0, 1, 0]), ([7, 3], [-1, 0])]
        host = [torch.from_numpy(rng.random(s, np.float32).clip(1e-6, 0.999)) for s in ((6, V), (6,), (2, V))]
        host[0] /= host[0].sum(1, keepdim=True)
        host[1][1] = 1e-6                               # node 1 is taken
        pinned = [h.pin_memory() for h in host]
        m.decode_tree(tree)
        lg = torch.from_numpy(m.logits(6)).cuda()
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
        path, n_path, nxt = binding.op_verify_tree(lg, i32([5, 9, 11, 2, 7, 3]), i32([-1, 0, 1, 0, -1, 0]), i32([0, 4, 6]),
                                                   64, 0.9, *[h.cuda() for h in host])
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            made = [torch.full_like(h, 0.5, device="cuda") for h in host]
            torch.cuda._sleep(100_000_000)              # (some 50 ms)
            for t, h in zip(made, pinned):
                t.copy_(h, non_blocking=True)
            got = m.accept_tree(0.9, *made)
        toks = [[5, 9, 11, 2], [7, 3]]
        assert got == [[toks[b][i] for i in path[b, 1:n_path[b]].tolist()] + [nxt[b].item()] for b in range(2)]
        m.decode_tree([([got[0][-1]], [-1])])
        with pytest.raises(ValueError):
            m.accept_tree(0.9, None, host[1][:1], host[2][:1])
        m.accept_tree()
    finally:
        m.close()
