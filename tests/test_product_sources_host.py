"""What a run of the product kernels cannot show: the scopes of their barrier
operations, read from the sources (no GPU).

A release orders a thread's writes for the observers inside its scope only.  An
arrival at another CTA's barrier is therefore relaxed at cluster scope, behind a
release fence of that scope where it hands over written memory; and who waits
for such an arrival has an acquire fence of that scope behind the wait."""
import os
import re

from norm_activation_fp8_gb300 import build

REMOTE = "mbar_arrive_cluster_written"


def sources():
    for name in sorted(os.listdir(build.CSRC)):
        if name.endswith((".cu", ".cuh")):
            with open(os.path.join(build.CSRC, name)) as f:
                yield name, re.sub(r"//[^\n]*", "", f.read())


def body(text, head):
    """The braces behind ``head``."""
    at = text.index("{", text.index(head))
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at:i + 1]
    raise AssertionError(head)


def test_arrivals_at_other_ctas_have_cluster_scope():
    found = 0
    for name, text in sources():
        for op in re.findall(r"mbarrier\.arrive[\w.:]*shared::cluster[\w.:]*", text):
            found += 1
            assert ".relaxed.cluster." in op or ".release.cluster." in op, (name, op)
    assert found >= 1
    hand_over = body(dict(sources())["tcgen05.cuh"], f"void {REMOTE}")
    fence = re.search(r"fence\.release[\w.:]*\.cluster;", hand_over)
    assert fence and fence.start() < hand_over.index("mbar_arrive_cluster(")


def test_waits_for_written_memory_acquire_at_cluster_scope():
    """Every wait, and every look ahead, at a barrier on which another CTA's threads
    hand over what they have written."""
    files = dict(sources())
    tma, common = files["tma.cuh"], files["gemm_common.cuh"]
    waits = re.findall(r"try_wait\.parity([\w.]*)\.shared::cta", body(tma, "bool mbar_try_wait"))
    assert waits == [".relaxed.cluster", ""]  # CLUSTER, otherwise
    looks = re.findall(r"test_wait\.parity([\w.]*)\.shared::cta\.b64 vg_look(\d)", body(tma, "void mbar_look"))
    assert looks == [("", "0"), (".relaxed.cluster", "1")]
    assert re.search(r"fence\.acquire[\w.:]*\.cluster;", body(tma, "void acquire_cluster_written"))
    wait = body(common, "bool warp_wait_phase(bool seen")
    assert wait.index("wait_phase<CLUSTER>") < wait.index("if constexpr (CLUSTER) acquire_cluster_written();")
    seen = 0
    for name, text in files.items():
        for bar in set(re.findall(REMOTE + r"\(cluster_addr\(&sm\.(\w+)", text)):
            calls = re.findall(r"(warp_wait_phase|wait_phase|mbar_wait_bounded|mbar_try_wait|mbar_look)"
                               r"(<\w+>)?\((\w+, )?&sm\." + bar + r"\b", text)
            assert {x[0] for x in calls} == {"warp_wait_phase", "mbar_look"}, (name, bar)
            for call, kind, look in calls:
                assert kind == "<1>" if call == "mbar_look" else (kind == "<true>" and look), (name, bar, call)
            seen += 1
    assert seen >= 1
