"""cg_rotate at the number of heads from which four of a row go to a lane group, 8192 of all rows, and just above."""
import pytest

from test_gpu_rotate import Rot

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("B,n,Hq,H", [(1, 1024, 6, 2), (1, 1, 8191, 1), (1, 1, 8192, 1), (1, 1025, 6, 2), (3, 911, 2, 1), (2, 1025, 3, 1),
                                      (1, 911, 8, 1), (1, 2731, 2, 1), (1, 2048, 3, 1), (1, 2049, 3, 1)])
def test_one_head_or_four_to_a_lane_group(B, n, Hq, H, bf16):
    r = Rot(110 + n, B=B, n=n, Hq=Hq, H=H, bf16=bf16)
    r.check(r.run())


def test_both_forms_give_the_same_bits():
    """A row's result does not depend on how many others go with it."""
    t = __import__("torch")
    r = Rot(120, B=1, n=2048, Hq=6, H=2)
    q, k = r.run()
    few = Rot(120, B=1, n=2048, Hq=6, H=2)
    few.n = 300
    few.starts = r.starts
    qo, ko = few.run(r.q[:, :300].contiguous(), r.k[:, :300].contiguous(), t.empty_like(r.q[:, :300]), t.empty_like(r.k[:, :300]))
    assert t.equal(qo, q[:, :300]) and t.equal(ko, k[:, :300])
