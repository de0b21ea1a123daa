"""What the binding of the 8-bit and windowed operations looks at before it calls the library: CPU only."""
import pytest

from flow_matching_mmdit_b200 import binding

torch = pytest.importorskip("torch")

BAD, SHAPE = 1, 2
D = 128


def refused(status, call):
    with pytest.raises(binding.LensError) as e:
        call()
    assert e.value.status == status


def rows(x, samples, mod_stride, d=D):
    return binding._rows("norm", x.get_device(), x, samples, d, mod_stride)


def test_modulation_rows_have_to_be_at_the_stated_distance():
    mod = torch.zeros(4, 3, D)
    for view in (mod[:, 1], mod[:, 1:2], mod[None, :, 1], mod[:, 2], mod.view(4, 3 * D)[:, D:]):
        assert rows(view, 4, 3 * D) == view.data_ptr()
    refused(SHAPE, lambda: rows(mod[:, 1], 4, D))             # rows between the view's own
    refused(SHAPE, lambda: rows(mod[:, 1], 5, 3 * D))         # one sample too many
    refused(SHAPE, lambda: rows(mod[:2, 1], 3, 3 * D))
    # separate tensors with the distance of a common one would be read past their ends
    alone = torch.zeros(4, D)
    refused(SHAPE, lambda: rows(alone, 4, 3 * D))
    refused(SHAPE, lambda: rows(alone, 2, 3 * D + 4))
    assert rows(alone, 4, D) == alone.data_ptr()


def test_modulation_rows_of_one_sample_and_of_flat_tensors():
    flat = torch.zeros(4 * 3 * D)
    assert rows(flat[D:], 4, 3 * D) == flat.data_ptr() + 4 * D          # from a start inside the buffer
    assert rows(flat.view(12, D)[1:], 4, 3 * D) == flat.data_ptr() + 4 * D
    refused(SHAPE, lambda: rows(flat[2 * D + 1:], 4, 3 * D))
    one = torch.zeros(D)
    assert rows(one, 1, 3 * D) == rows(one, 7, 0) == one.data_ptr()     # one row for every sample
    assert rows(one.view(2, D // 2), 1, 0) == one.data_ptr()
    refused(SHAPE, lambda: rows(one, 2, D))
    refused(SHAPE, lambda: rows(one[:-16], 1, 0))
    refused(SHAPE, lambda: rows(torch.zeros(2, D)[:, :-16], 2, D))


@pytest.mark.parametrize("at", [0, 1])
@pytest.mark.parametrize("value", [2 ** 31, -2 ** 31 - 1, 2 ** 70])
def test_lengths_past_32_bits_are_refused(at, value):
    lengths = [[0, 0], [8, 8]]
    lengths[at][1] = value
    refused(BAD, lambda: binding.lens_op_attention_window(None, None, None, 2, 4, 4, 1, 8, *lengths, 1, 0, 0, 0.125, None,
                                                          stream=0))
