"""The key-value cache on the GPU where a caller's data are at the edge of what it may hold: tables whose pages
the references call free.
"""
import numpy as np
import pytest
import torch

import gated_delta_rule_deltanet_gb300 as kda
from gated_delta_rule_deltanet_gb300 import _lib
from oracle import cache as oc

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def ints(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def no_error():
    torch.cuda.synchronize()
    assert kda.get_device_error() == 0


def error():
    torch.cuda.synchronize()
    return kda.get_device_error()


# ------------------------------------------------------------------------------------------ tables

def refused(table, lens, refs, parent, new, P):
    got = kda.cache_update(ints(table), ints(lens), ints(refs), None if parent is None else ints(parent), ints(new), page_size=P)
    assert error() == _lib.KDA_DEVERR_PAGE
    assert torch.all(got.table == -1) and not got.lens.any() and not got.kept.any()
    assert torch.equal(got.refs, ints(refs)) and torch.all(got.src == -1) and torch.all(got.dst == -1)
    no_error()


@pytest.mark.parametrize("parent,new,free", [
    ([0, 0, 1], [7, 6, 6], 0),                 # a full page that both continuations of its row share
    ([0, 1, 1], [7, 6, 6], 2),
    ([0, 1, 1, 1], [8, 6, 6, 5], 2),
    ([0, 0, 0, 1], [8, 8, 3, 5], 1),           # full for two of them, not kept by the third
    ([0, 0, 1], [7, 6, 6], 1),                 # the page that they end inside
    ([0, 1], [8, 5], 3),                       # rows that only go on
    ([-1, 1, 1], [4, 5, 5], 0),                # a row that ends
])
def test_update_refuses_a_free_page_of_any_row(parent, new, free):
    refs = np.array([1, 1, 1, 1, 0, 0, 0, 0, 0, 0], np.int32)
    refs[free] = 0
    refused(np.array([[0, 1], [2, 3]], np.int32), [8, 5], refs, parent, new, 4)


@pytest.mark.parametrize("S", [4096, 4097, 6000])
@pytest.mark.parametrize("fork", [False, True])
@pytest.mark.parametrize("page", [0, 1])
def test_update_refuses_a_free_page_of_many_rows(S, fork, page):
    """One row of thousands names a free page; page 0 of it is full, page 1 the one that it ends inside."""
    table = np.arange(2 * S, dtype=np.int32).reshape(S, 2)
    refs = np.concatenate([np.ones(2 * S), np.zeros(50)]).astype(np.int32)
    parent = np.arange(S)
    if fork:
        parent[5] = 17
    new = np.full(S, 6)
    got, ref = kda.cache_update(ints(table), ints([5] * S), ints(refs), ints(parent), ints(new), page_size=4), \
        oc.update(table, [5] * S, refs, parent, new, 4)
    no_error()
    assert np.array_equal(got.table.cpu().numpy(), ref[0]) and np.array_equal(got.refs.cpu().numpy(), ref[2])
    refs[table[17, page]] = 0
    refused(table, [5] * S, refs, parent, new, 4)
