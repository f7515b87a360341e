"""tf_fork_seq: a forked sequence goes on exactly as its source would, on caches of its own."""
import numpy as np
import pytest
import torch

from dual_ar_decode_gb300 import Decoder, TfError
from synth import TINY, make_prompt, make_weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


@pytest.fixture(scope="module")
def weights():
    return make_weights(TINY, seed=51)


def decoder(weights, paged, dims=TINY, slots=4):
    dec = Decoder(dims, "bf16", max_batch=slots, paged=paged)
    dec.load_weights(weights)
    return dec


# positions after the prompt's ids and the frames before the fork: inside a page, at its end, and just begun
@pytest.mark.parametrize("P,before", [(10, 3), (31, 1), (32, 0), (33, 0), (1, 0), (40, 2), (30, 3)])
@pytest.mark.parametrize("paged", [False, True])
def test_a_fork_decodes_what_its_source_does(weights, paged, P, before):
    """Greedy and forced alike in both slots: the fork's logits equal the source's bit for bit, and neither changes
    what the source had emitted without a fork."""
    prompt = make_prompt(TINY, P, seed=P)[0]
    other = make_prompt(TINY, 7, seed=99)[0]
    alone = decoder(weights, paged)
    alone.prefill_seq(0, prompt)
    alone.prefill_seq(2, other)
    want = [alone.decode_frame(logits=True) for _ in range(before + 5)]
    alone.close()
    dec = decoder(weights, paged)
    dec.prefill_seq(0, prompt)
    dec.prefill_seq(2, other)
    for t in range(before):
        dec.decode_frame()
    dec.fork_seq(0, 1)
    for t in range(before, before + 5):
        f, z = dec.decode_frame(logits=True)
        assert np.array_equal(f[0], want[t][0][0]) and np.array_equal(f[2], want[t][0][2])
        assert np.array_equal(f[1], f[0])
        assert np.array_equal(z[1].view(np.uint32), z[0].view(np.uint32))
        assert np.array_equal(z[0].view(np.uint32), want[t][1][0].view(np.uint32))
    dec.close()


@pytest.mark.parametrize("paged", [False, True])
def test_forks_part_when_they_are_fed_different_ids(weights, paged):
    """After the fork each slot writes rows of its own: fed different ids, each goes where a sequence fed those ids
    from the start goes."""
    prompt = make_prompt(TINY, 20, seed=3)[0]
    rng = np.random.default_rng(0)
    ids = rng.integers(0, TINY.codebook_size, (14, 3, 10)).astype(np.int32)
    ids[:4] = ids[:4, :1]                                    # the same past
    refs = []
    for b in range(3):
        dec = decoder(weights, paged)
        for s in range(3):
            dec.prefill_seq(s, prompt)
        refs.append([dec.decode_frame(forced=np.repeat(ids[t, b:b + 1], 3, 0), logits=True)[1][b] for t in range(14)])
        dec.close()
    dec = decoder(weights, paged)
    dec.prefill_seq(2, prompt)
    for t in range(4):
        z = dec.decode_frame(forced=ids[t], logits=True)[1]
        assert np.array_equal(z[2].view(np.uint32), refs[2][t].view(np.uint32))
    dec.fork_seq(2, 0)
    dec.fork_seq(0, 1)                                       # a fork of a fork
    for t in range(4, 14):                                   # over a page's end
        z = dec.decode_frame(forced=ids[t], logits=True)[1]
        for b in range(3):
            assert np.array_equal(z[b].view(np.uint32), refs[b][t].view(np.uint32)), (t, b)
    dec.close()


def test_shared_pages_come_back_when_the_last_holder_leaves(weights):
    """Forks over forks, released in every order: each time all slots can still be filled to the last position."""
    d = TINY.replace(max_seq_len=96)
    dec = decoder(weights, True, dims=d, slots=3)
    for order in ([0, 1, 2], [2, 1, 0], [1, 0, 2]):
        dec.prefill_seq(0, make_prompt(d, 70, seed=1)[0])
        dec.fork_seq(0, 1)
        dec.fork_seq(1, 2)
        dec.fork_seq(0, 2)                                   # over an occupied slot
        dec.decode_frames(3)
        for s in order:
            dec.release_seq(s)
    for s in range(3):
        dec.prefill_seq(s, make_prompt(d, 90, seed=s)[0])
    assert dec.decode_frames(7).shape == (7, 3, 10)          # positions 89 .. 95: every page in use
    with pytest.raises(TfError, match="CAPACITY"):
        dec.decode_frame()
    dec.close()


def test_a_forks_draws_use_its_own_slot_and_its_repetition_window(weights):
    """Takes of one prompt: the fork draws as a sequence that had always been in that slot would."""
    s = {"top_k": 8, "seed": 5, "rep_window": 6, "rep_penalty": 1.3}
    prompt = make_prompt(TINY, 12, seed=3)[0]
    forced = np.random.default_rng(1).integers(0, TINY.codebook_size, (4, 2, 10)).astype(np.int32)
    forced[:, 1] = forced[:, 0]
    both = decoder(weights, True, slots=2)
    for b in range(2):
        both.prefill_seq(b, prompt)
    for t in range(4):
        both.decode_frame(s, forced=forced[t])
    want = [both.decode_frame(s)[0] for _ in range(4)]
    both.close()
    dec = decoder(weights, True, slots=2)
    dec.prefill_seq(0, prompt)
    dec.prefill_seq(1, prompt)                               # (so that both runs take the batched kernels)
    for t in range(4):
        dec.decode_frame(s, forced=forced[t])
    dec.fork_seq(0, 1)
    got = [dec.decode_frame(s)[0] for _ in range(4)]
    dec.close()
    assert np.array_equal(np.stack(got), np.stack(want))
    assert not np.array_equal(np.stack(got)[:, 0], np.stack(got)[:, 1])


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("T,P", [(50, 33), (24, 24), (33, 33), (96, 64)])
def test_forks_with_caches_of_other_lengths(weights, paged, T, P):
    """Slabs that 32 rows do not divide, and a sequence whose cache is full."""
    d = TINY.replace(max_seq_len=T)
    dec = decoder(weights, paged, dims=d, slots=3)
    prompt = make_prompt(d, P, seed=P)[0]
    dec.prefill_seq(0, prompt)
    dec.decode_frame()
    dec.fork_seq(0, 2)
    for _ in range(min(4, T - P)):
        f, z = dec.decode_frame(logits=True)
        assert np.array_equal(z[0].view(np.uint32), z[2].view(np.uint32)) and (f[1] == -1).all()
    if T - P < 4:
        with pytest.raises(TfError, match="CAPACITY"):
            dec.decode_frame()
    dec.close()


def test_a_fork_of_a_lockstep_batch_of_one(weights):
    """After tf_prefill the one sequence runs on the batch-1 kernels, and with its fork on the batched ones."""
    dec = decoder(weights, True)
    dec.prefill(make_prompt(TINY, 11, seed=2))
    dec.decode_frame()
    dec.fork_seq(0, 3)
    for _ in range(3):
        f, z = dec.decode_frame(logits=True)
        assert f.shape == (4, 10) and (f[1:3] == -1).all()
        assert np.array_equal(f[0], f[3]) and np.array_equal(z[0].view(np.uint32), z[3].view(np.uint32))
    dec.release_seq(0)
    f, _ = dec.decode_frame()
    assert (f[:3] == -1).all() and (f[3] >= 0).all()
    dec.close()


def test_fork_errors(weights):
    dec = decoder(weights, True, slots=2)
    dec.prefill_seq(0, make_prompt(TINY, 4)[0])
    for src, dst in ((0, 0), (0, 2), (-1, 0), (2, 0), (0, -1)):
        with pytest.raises(TfError, match="INVAL"):
            dec.fork_seq(src, dst)
    with pytest.raises(TfError, match="STATE"):
        dec.fork_seq(1, 0)
    f, _ = dec.decode_frame()
    assert f.shape == (1, 10)                                # nothing changed
    dec.close()
