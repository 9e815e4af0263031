"""The ordering rules of the adapter kernels, read from their sources (no GPU needed): each is one
whose breach could lose a value or leave a kernel waiting only now and then, so that no run
shows it reliably."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "int8_quantized_linear_q8_b200", "csrc")


def _code(name):
    """The file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _body(text, name):
    """The body of the function `name`, braces matched."""
    at = re.search(r"\b%s\s*\([^;{]*?\)\s*\{" % name, text, re.S).end()
    depth, end = 1, at
    while depth:
        depth += {"{": 1, "}": -1}.get(text[end], 0)
        end += 1
    return text[at:end]


def _first(body, words):
    found = [body.find(w) for w in words if w in body]
    return min(found) if found else None


BARRIER = ("barrier.cluster.wait", "cluster_sync_all(", "lt_cluster_sync(")
PEER = ("st.shared::cluster", "ld.shared::cluster", "cluster_sum4(", "lt_arrive(", "lt_tma_pair(",
        "lt_commit(")


@pytest.mark.parametrize("source,kernel", [("k_lora_decode.cu", "k_lora_decode"),
                                           ("k_lora.cu", "k_lora_shrink"),
                                           ("k_lora.cu", "lora_grad_tile"),
                                           ("k_lora_tc.cu", "k_lora_tc")])
def test_a_cluster_has_started_before_its_shared_memory_is_used(source, kernel):
    """Another CTA's shared memory may be touched once that CTA is known to run: behind a
    cluster barrier."""
    body = _body(_code(source), kernel)
    barrier, peer = _first(body, BARRIER), _first(body, PEER)
    assert peer is not None and barrier is not None
    assert barrier < peer


def test_a_warp_goes_on_from_a_wait_as_one():
    """A wait that runs out may do so for some lanes of a warp and not for others, so what
    follows (shuffles, warp barriers, tensor-memory reads, which need the whole warp) goes by a
    vote."""
    body = _body(_code("k_lora_tc.cu"), "k_lora_tc")
    waits = [m.start() for m in re.finditer(r"\bmbar_wait\(", body)]
    assert len(waits) >= 9
    for at in waits:
        statement = body[max(body.rfind(c, 0, at) for c in ";{}"):at]
        assert "__all_sync(0xffffffffu," in statement, body[at - 120:at + 80]


def test_both_ctas_of_a_pair_see_the_last_commit():
    """The issuer's commits arrive in both CTAs' shared memory some time after it leaves, so
    each CTA waits for the last of them, the first one before its tensor memory is read and the
    other one before it ends."""
    body = _body(_code("k_lora_tc.cu"), "k_lora_tc")
    assert "lt_commit(mma_done, both)" in body
    last_sync = body.rfind("lt_cluster_sync();")
    tail = body[last_sync:]
    drain, dealloc = tail.find("mbar_drain(mma_done, 0, status)"), tail.find("tcgen05.dealloc")
    assert 0 < drain < dealloc
    # not under a condition on the CTA's rank
    assert "rank" not in tail[:drain]


@pytest.mark.parametrize("source", ["k_checkpoint.cu", "k_lora_decode.cu", "k_lora.cu"])
def test_what_the_kernel_before_writes_is_not_read_as_constant(source):
    """These kernels start while the one before them still writes what they read, so none of
    their loads may promise memory that does not change while they live (ld.global.nc)."""
    text = _code(source)
    assert "griddepcontrol.wait" in text
    assert not re.findall(r"\bldg_\w+|\b__ldg\b|global\.nc", text)
