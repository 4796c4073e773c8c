"""More of what the operators around the epilogue refuse before any CUDA call (CPU only)."""
from tests.test_rows_refusals import bd, process  # noqa: F401


def test_process_refuses_mask_rows_without_words(bd):  # noqa: F811
    assert process(bd, mask=bd.dspark_mask_t(None, 4, 4, 64)) == 1
    assert process(bd, mask=bd.dspark_mask_t(None, 4, 4, None)) == 1


def test_process_refuses_list_lengths(bd):  # noqa: F811
    assert process(bd, history_nnz=-1) == 1
    assert process(bd, bias_nnz=-1) == 1


def test_process_refuses_misplaced_rows(bd):  # noqa: F811
    """The requests' parameters are bytes to torch: a slice of them may start anywhere."""
    for at in (257, 258, 259):
        assert process(bd, rows=at) == 1
