"""Fork and compaction on both sides of the sizes at which their launches change: one CTA or a cluster
for the counts, the tables in the plan's launch or in one of their own."""
import pytest
import torch

from tests.test_gpu_cache import Dev, _compact

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dsa_sparse_attention_gb300.build import build
    build()


# (rows, forks, stride): 1,024 table entries a CTA go with the plan
SIZES = [(300, 8, 128), (300, 5, 205), (300, 4, 300), (16384, 32, 32), (16385, 32, 32), (17000, 64, 128), (17000, 61, 135),
         (17000, 300, 60)]


@pytest.mark.parametrize("rows,n,stride", SIZES)
def test_fork_around_the_rules(rows, n, stride):
    bs = 16
    lens = [bs * (stride - 1) + 3, bs * 20, 1]
    d = Dev(rows, [min(L, bs * (rows // 3)) for L in lens] + [0] * n, bs=bs, seed=rows + n, stride=stride)
    want = [i % 3 for i in range(n)]
    src, dst = d.fork(want, [3 + i for i in range(n)])
    d.copy(src, dst)
    d.free([3 + i for i in range(0, n, 2)])
    _compact(d, False)
    d.check()
    _compact(d, True)
    d.check()
    assert sum(1 for v in d.plain.ref if v) == max(i for i, v in enumerate(d.plain.ref) if v) + 1


@pytest.mark.parametrize("reqs,stride", [(8, 128), (5, 205), (64, 128), (61, 135)])
@pytest.mark.parametrize("rows", [900, 17000])
def test_compact_around_the_rules(rows, reqs, stride):
    bs = 16
    lens = [bs * (7 * i % 13) + i for i in range(reqs)]
    d = Dev(rows, lens, bs=bs, seed=reqs, stride=stride, extra=17)
    d.free([i for i in range(0, reqs, 3)])
    for alias in (False, True):
        _compact(d, alias)
        d.check()
