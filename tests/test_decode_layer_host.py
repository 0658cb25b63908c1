"""The decoder's token places on the CPU: inside the table, at its end and past it."""
import pytest
import torch

from moe_decode_expert_gb300.decode_layer import Decoder, full_width, places


@pytest.mark.parametrize("page", [1, 7, 16])
@pytest.mark.parametrize("pages", [1, 3])
def test_places_at_the_end_of_the_table(page, pages):
    n = page * pages
    pos = torch.tensor([0, n - 1, n, n + 1, n + 1000, 2 ** 31 - 1, 2 ** 40, -1, -2, -(2 ** 40)])
    g = torch.Generator().manual_seed(n)
    table = torch.randperm(len(pos) * pages, generator=g).view(len(pos), pages).to(torch.int32)
    before = pos.clone()
    slots, lens = places(pos, table, page)
    assert slots.dtype is torch.int64 and lens.dtype is torch.int32 and torch.equal(pos, before)
    assert slots[0] == table[0, 0] * page and slots[1] == table[1, -1] * page + page - 1
    assert (slots[2:] == -1).all()  # nothing is stored
    # lengths: right inside, past the table (which is recorded) beyond, none before
    assert lens[:2].tolist() == [1, n] and (lens[2:7] == n + 1).all()
    assert lens[7] == 0 and (lens[8:] == -1).all()


def test_places_inside_the_table():
    page, pages = 5, 4
    pos = torch.arange(20)
    table = torch.randperm(80).view(20, 4).to(torch.int32)
    slots, lens = places(pos, table, page)
    for i in range(20):
        assert slots[i] == int(table[i, i // page]) * page + i % page and lens[i] == i + 1


@pytest.mark.parametrize("layers,batch,max_len", [([], 1, 16), ([{}], 0, 16), ([{}], 1, 0)])
def test_a_decoder_without_places_is_refused(layers, batch, max_len):
    with pytest.raises(ValueError):
        Decoder(full_width(), layers, batch, max_len, torch.device("cpu"))
