"""Workspace sizes of the gated product while another thread holds a test
override: the override is its thread's alone (host only)."""
import threading

from convolution_nhwc_amd import api


def size(op=api.OP_DGRAD, rows=300, c=64, f=96):
    forced = api._forced.key
    return api._gated_desc(forced, op, 0, rows, c, f, c, f, 0, api.BF16)[1]


def elsewhere(fn):
    out = []
    t = threading.Thread(target=lambda: out.append(fn()))
    t.start()
    t.join()
    return out[0]


def test_another_threads_override_does_not_change_sizes():
    free = size(rows=301)
    with api.override(tune=256, split_c=4):
        forced = size()
        # asked for the first time while the override is held, and asked again
        assert elsewhere(size) != forced
        assert elsewhere(lambda: size(rows=301)) == free
    assert size() == elsewhere(size) != forced


def test_an_override_in_another_thread_stays_there():
    inside, asked = threading.Event(), threading.Event()
    got = []

    def hold():
        with api.override(tune=256, split_c=4):
            got.append(size(rows=302))
            inside.set()
            asked.wait(30)
            got.append(size(rows=302))
    t = threading.Thread(target=hold)
    t.start()
    assert inside.wait(30)
    free = size(rows=302)
    asked.set()
    t.join()
    assert got[0] == got[1] != free


def test_nested_calls_after_an_override_use_the_free_sizes():
    with api.override(tune=128, split_c=5):
        forced = size(rows=303)
    assert size(rows=303) != forced
    with api.override(tune=128, split_c=5):
        assert size(rows=303) == forced
