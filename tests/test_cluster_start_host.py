"""Kernels that run in clusters, read as text: a CTA's shared memory may be written, and its barriers be signalled, by another
CTA of the cluster only once that CTA has begun to run, so every kernel's first remote access stands behind a wait for the
cluster's barrier."""
import pathlib
import re

import pytest

CSRC = pathlib.Path(__file__).resolve().parents[1] / "transformer_fwd_bwd_gb300" / "csrc"
# stores, arrivals and addresses in another CTA; copies that complete on another CTA's barrier
REMOTE = re.compile(r"st\.shared::cluster|mapa\.shared::cluster|mapa_shared\(|mbar_arrive_cluster\(|cluster_store\(|tma_load_4d_pair\(|tma_load_4d_mc\(")
WAIT = re.compile(r"barrier\.cluster\.wait|cluster_sync_all\(\)|cluster_barrier\(\)")


def kernels(text):
    """(name, body) of every __global__ function, comments taken out."""
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    text = re.sub(r"//[^\n]*", "", text)
    for m in re.finditer(r"__global__", text):
        at = text.index("{", m.end())
        depth, end = 0, at
        while True:
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            end += 1
            if depth == 0:
                break
        yield text[m.end():at], text[at:end]


def remote_kernels():
    for path in sorted(CSRC.glob("*.cu*")):
        for head, body in kernels(path.read_text()):
            if REMOTE.search(body):
                yield path.name, re.findall(r"(\w+_kernel)\b", head)[-1], body


def test_the_kernels_are_found():
    names = {n for _, n, _ in remote_kernels()}
    assert {"embedding_sort_kernel", "token_logprobs_kernel", "muon_product_kernel", "gemm_kernel", "ce_split_kernel"} <= names


@pytest.mark.parametrize("file,name,body", [pytest.param(*k, id=k[1]) for k in remote_kernels()])
def test_cluster_has_started_before_the_first_remote_access(file, name, body):
    wait = WAIT.search(body)
    assert wait and wait.start() < REMOTE.search(body).start(), f"{file}: {name}"
