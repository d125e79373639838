"""CPU check of the kernels' sources: no CTA of a cluster writes into another's shared memory before that one is known to have begun.

A CTA's shared memory may be written from outside only once the CTA runs, which a barrier of the cluster that all its CTAs came to shows.
Such a race cannot be provoked safely, so the order is held to where it stands: in the text.
"""
import os
import re

import pytest

from gated_delta_rule_23_gb300 import _native

SENDS = re.compile(r"st\.shared::cluster|store_cluster\(in_cta")
WAITS = re.compile(r"barrier\.cluster\.wait|cluster_sync\(\);")


def kernels():
    for path in _native.SOURCES:
        text = open(path).read()
        starts = [m.start() for m in re.finditer(r"__global__", text)] + [len(text)]
        for i, (a, b) in enumerate(zip(starts, starts[1:])):
            if SENDS.search(text[a:b]):
                yield pytest.param(text[a:b], id=f"{os.path.basename(path)}-{i}")


def test_there_are_such_kernels():
    assert len(list(kernels())) >= 3


@pytest.mark.parametrize("body", list(kernels()))
def test_a_cluster_has_begun_before_its_ctas_write_to_each_other(body):
    wait = WAITS.search(body)
    assert wait and wait.start() < SENDS.search(body).start()
