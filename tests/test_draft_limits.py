"""Trees of more drafts than the masks have bits: attended as chains, accepted as chains."""
import pytest
import torch

from tests import drafts_ref as ref
from tests.test_abi import FAKE
from tests.test_paged_abi import lib  # noqa: F401

I32 = torch.int32


def test_refusals(lib):  # noqa: F811
    import sequence_attn_fwd_gb300 as sa

    def accept(words=1, parents=FAKE, path=FAKE, B=2, total=5):
        return lib.draft_accept_words(parents, FAKE, FAKE, FAKE, None, path, FAKE, FAKE, B, total, words, None)

    assert accept(words=5) == 2 and accept(words=-1) == 1 and accept(parents=0) == 1 and accept(path=0) == 1
    assert accept(B=4097) == 2 and accept(B=0) == 0 and accept(total=-1) == 1
    i = lambda *x: torch.tensor(x, dtype=I32)  # noqa: E731
    args = i(-1, 0, 1), i(0, 3), i(1, 2, 3), i(1, 2, 3)
    for bad in (torch.zeros((3, 1), dtype=I32), torch.zeros((2, 1), dtype=torch.int64), torch.zeros(3, dtype=torch.int64)):
        with pytest.raises(ValueError, match="int64"):
            sa.draft_accept(*args, tree=bad)
    for words in (0, 5):
        with pytest.raises(ValueError, match="words"):
            sa.draft_accept(*args, tree=torch.zeros((3, words), dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA"):
        sa.draft_accept(*args, tree=torch.zeros((3, 1), dtype=torch.int64))


@pytest.mark.gpu
@pytest.mark.parametrize("words", [1, 2, 3, 4])
@pytest.mark.parametrize("with_given", [False, True])
def test_a_tree_that_was_attended_as_a_chain_is_accepted_as_one(cuda_dev, words, with_given):
    import sequence_attn_fwd_gb300 as sa

    g = torch.Generator().manual_seed(words)
    most = 64 * words
    sizes = [most, most + 1, 300, 0, 9, 1500, 2600, 65, 1]
    trees = [[-1] + [int(torch.randint(0, t, (), generator=g)) for t in range(1, n)] if n else [] for n in sizes]
    cu = [0]
    for n in sizes:
        cu.append(cu[-1] + n)
    dev = lambda x: torch.tensor(x, dtype=I32, device=cuda_dev)  # noqa: E731
    parents, offsets = dev([p for x in trees for p in x]), dev(cu)
    masks, depths = sa.draft_tree(parents, offsets, words)
    given = [1, 3, 300, 2, 9, 1, 1200, 64, 5] if with_given else [1] * len(sizes)
    meant = [[t - 1 for t in range(len(x))] if len(x) > most else x for x in trees]
    for chosen in (1, 2):
        tokens, choices = (torch.randint(0, chosen, (cu[-1],), generator=g).tolist() for _ in range(2))
        args = parents, offsets, dev(tokens), dev(choices), dev(given) if with_given else None
        got = sa.draft_accept(*args, tree=masks)
        want = ref.accept(meant, tokens, choices, given)
        assert [x.tolist() for x in got] == list(want)
        # the places of the kept tokens follow each other where the attention took them as a chain
        for b, n in enumerate(sizes):
            if n > most:
                line = got[0][cu[b]:cu[b] + int(got[1][b])].tolist()
                assert line == list(range(len(line))) and depths[cu[b]:cu[b + 1]].tolist() == list(range(n))
        free = sa.draft_accept(*args)
        want = ref.accept(trees, tokens, choices, given)
        assert [x.tolist() for x in free] == list(want)
