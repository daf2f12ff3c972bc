"""The kernel files' error words: each that a wait can set is read and cleared by ``device_error``. No wait runs out here: the host
sets a word (FXTX_PLANT_ERROR)."""
import os
import re

import pytest
import torch

import dense_linear_algebra_gb300 as fx

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dense_linear_algebra_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def words():
    """What ``take_errors`` reads, by the names of the files' functions."""
    listed = re.search(r"const ErrorWords w = \{\{(.*?)\}\}", source("api.cu"), re.S).group(1)
    return re.findall(r"(\w+)_error_word\(\)", listed)


def test_the_words_of_the_files():
    names = words()
    assert len(set(names)) == len(names) == int(re.search(r"kErrorWords = (\d+)", source("api.cu")).group(1))
    exported = [m.group(1) for f in sorted(os.listdir(CSRC)) if f.endswith(".cu")
                for m in re.finditer(r"int\* (\w+)_error_word\(\) \{", source(f))]
    assert sorted(exported) == sorted(names)


def test_each_file_that_waits_has_its_word():
    """A file has a word of its own: one that waits, by itself or by the kernels of a header, has to give it out."""
    waits = re.compile(r"mbar_wait_bounded\(|tc_wait\(|warp_wait\(|raise_error\(|#include \"product_(tc|split)\.cuh\"")
    for f in sorted(os.listdir(CSRC)):
        if f.endswith(".cu") and waits.search(source(f)):
            assert "_error_word() { return device_error_word(); }" in source(f), f


@pytest.mark.gpu
def test_each_word_is_read_and_cleared(monkeypatch):
    assert fx.device_error() == fx.FXTX_OK
    side = torch.cuda.Stream()
    for i in range(len(words())):
        monkeypatch.setenv("FXTX_PLANT_ERROR", str(i))
        assert fx.device_error(side if i % 2 else None) == fx.FXTX_ERR_TIMEOUT, words()[i]
        monkeypatch.delenv("FXTX_PLANT_ERROR")
        assert fx.device_error() == fx.FXTX_OK, words()[i]
