"""What the serving-step kernels must have in their source and no run can show for certain: the order of
barriers and of stores into other blocks' shared memory. No GPU."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "weight_only_groupwise_gb300", "csrc")


def body(name: str, kernel: str) -> str:
    """A kernel's body, without comments."""
    text = open(os.path.join(CSRC, name)).read()
    text = re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", text, flags=re.S))
    at = text.index("{", text.index(")", text.index(kernel + "(const")))
    depth = 0
    for end in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[end], 0)
        if depth == 0:
            return text[at:end]
    raise AssertionError("unbalanced braces")


def without_lambda(text: str, name: str) -> str:
    at = text.index(f"auto {name} = [&]")
    start = text.index("{", at)
    depth = 0
    for end in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[end], 0)
        if depth == 0:
            return text[:at] + text[end + 1:]
    raise AssertionError("unbalanced braces")


def test_sampling_blocks_know_that_their_cluster_runs_before_the_first_remote_access():
    text = body("nq_sample.cu", "sample_kernel")
    # the two helpers that store into other blocks count where they are called, not where they are defined
    for helper in ("exchange", "cluster_max"):
        text = without_lambda(text, helper)
    remote = min(m.start() for m in re.finditer(r"map_shared_rank|\bexchange\(|\bcluster_max\(|\bcl\.sync\(", text))
    wait = text.find("cluster_wait_begun()")
    arrive = text.find("cluster_begun()")
    assert 0 <= arrive < wait < remote
    assert text.count("cluster_begun()") == text.count("cluster_wait_begun()") == 1
    # every thread does both: under the same condition, at the kernel's outermost level, and nobody leaves between
    for at in (arrive, wait):
        assert text[:at].count("{") - text[:at].count("}") == 1
        assert text[:at].rstrip().endswith("if (C > 1)")
    assert "return" not in re.sub(r"\[&\]\([^)]*\) *\{.*?\};", "", text[arrive:wait], flags=re.S)


def test_paired_attention_publishes_zeroed_rows_at_cluster_scope():
    """Rows of V that the second block's softmax warps zero are read by the leading block's products: the arrival that
    tells the leader so releases at cluster scope, after every lane's stores."""
    text = body("nq_attn.cuh", "attn_kernel")
    helper = text[text.index("auto arrive_leader"):]
    helper = helper[:helper.index("};")]
    assert re.search(r"if \(lane == 0 && published\) mbar_arrive_remote\(", helper)
    calls = re.findall(r"\barrive_leader\(pready0 \+ 8 \* buf, (\w+)\)", text)
    assert calls == ["published"]
    # set where the zeros have been written, after the fence for the tensor cores' view of them, before the warp meets
    zeros = text[text.index("auto zero ="):]
    order = [zeros.index(x) for x in ("fence_proxy_async_smem();", "published = true;", "__syncwarp();", "arrive_leader(pready0")]
    assert order == sorted(order)


def test_no_attention_block_leaves_while_its_copies_are_on_their_way():
    """Any warp can give up waiting, also after the producers have asked for their last copies: they wait in any case, for the last
    into each slot, which is that of either of the two; the query tiles' warp for its last."""
    text = body("nq_attn.cuh", "attn_kernel")
    roles = text[text.index("if (warp == kAttnProducerK || warp == kAttnProducerV)"):]
    producer = roles[:roles.index("else if (PAIR && rank == 1 && warp == kAttnMma)")]
    assert "int* const mine = last_fill + (int)is_v * kAttnMaxSlots;" in producer and producer.count("if (lane < kSlots) mine[lane] = -1;") == 1
    loop = producer[producer.index("for (; w.more()"):]
    assert loop.index("__syncwarp();") < loop.index("tma_load_4d(") < loop.index("if (lane == 0) mine[slot] = seq;") < loop.index("id = id_next;")
    assert re.search(r"\}\s*named_bar_sync\(5, 64\);\s*const int last = lane < kSlots \? max\(last_fill\[lane\], last_fill\[kAttnMaxSlots \+ lane\]\) : -1;\s*"
                     r"if \(last >= 0\) mbar_wait_drain\(full0 \+ 8 \* lane, \(last / kSlots\) & 1, kDrainNs\);\s*\}\s*$", producer)
    assert text.count("named_bar_sync(5,") == 1 and "return" not in loop
    loader = roles[roles.index("else if (warp == kAttnLoader)"):]
    assert re.search(r"\}\s*if \(seg > 0\) mbar_wait_drain\(qfull, \(seg - 1\) & 1, kDrainNs\);\s*\} else \{", loader)
