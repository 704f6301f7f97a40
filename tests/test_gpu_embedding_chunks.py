"""GPU: the embedding gradient where its sorted tokens are cut into chunks of more than 16."""

import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_token_ops import TYPE_IDS, TYPES, test_embedding_grad as against_the_oracle  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import newton_schulz_momentum_gb300 as dm
    return dm


@pytest.mark.parametrize("kind", ["one", "distinct", "falling", "even"])
@pytest.mark.parametrize("dt", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("n,rows,dim", [(9001, 400, 4104), (20000, 30, 4104), (17003, 3000, 2056), (40001, 700, 1027)])
def test_long_chunks(dm, n, rows, dim, dt, kind):
    """Chunks of 32 and 64 tokens, with rows of 16-byte granules and without, and of either kind rows inside a chunk,
    across a few and across many of them."""
    against_the_oracle(dm, n, rows, dim, dt, kind)
