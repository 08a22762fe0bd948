"""Steps of many requests around the lengths where pa_linear_attention changes from the recurrent
form to the chunks, which depend on the head sizes and on how many states a step has."""
import pytest

from test_gpu_linear import run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv,d", [(2, 2, 128), (4, 2, 128), (16, 2, 128), (20, 2, 128), (3, 3, 64),
                                      (6, 3, 64)])
@pytest.mark.parametrize("requests", [3, 60])
def test_around_the_threshold(requests, hq, hkv, d):
    run([(7, 8, 9, 11, 12, 13, 15, 16, 17, 1, 0, 20)[i % 12] for i in range(requests)], hq, hkv, d,
        seed=requests, pad=3, fresh=(1,), drop=(2,))
    run([12] * requests, hq, hkv, d, seed=hq, decay="head", in_place=True)


def test_short_rows_alone():
    """No request is long, but the step has more tokens than a request may have of the short form."""
    run([16] * 100, 1, 1, 128, seed=1)
    run([12] * 60, 8, 2, 128, seed=2)
    run([2] * 7, 4, 2, 64, seed=3)
