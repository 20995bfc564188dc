"""CPU-only: outputs and workspaces of the linear layer, the top logits and the
distillation that share memory with an input are refused before any device
work."""

import pytest

import weighted_model_update_amd as fa
from test_learn_cpu import ARG, at, backward, distill, forward, topk


def refused(rc, word):
    assert rc == ARG
    assert word in fa.load().fedavg_last_error(), fa.load().fedavg_last_error()


TL = (at(12), at(13))
# R = 3 rows: 12 bytes of row weights, normalisers and losses, 60 and 72 of lists
INPUTS = {"row_weight": at(6, 8), "first list": at(1, 56), "second list": at(2, 68), "first values": at(3), "second values": at(4, 36),
          "first normaliser": at(12, 4), "second normaliser": at(13, 8)}


@pytest.mark.parametrize("name", list(INPUTS))
@pytest.mark.parametrize("which", ["loss", "lse", "dz", "err", "ws"])
def test_distill_loss_outputs_off_the_row_inputs(which, name):
    # a workspace has to start on 16 bytes
    p = INPUTS[name] if which != "ws" else at(INPUTS[name].value - (1 << 40) >> 36)
    refused(distill(True, tl=TL, **{which: p}), b"overlap")


@pytest.mark.parametrize("name", list(INPUTS))
@pytest.mark.parametrize("which", ["dz", "err", "ws"])
def test_distill_backward_outputs_off_the_row_inputs(which, name):
    p = INPUTS[name] if which != "ws" else at(INPUTS[name].value - (1 << 40) >> 36)
    refused(distill(False, tl=TL, **{which: p}), b"overlap")


@pytest.mark.parametrize("loss_call", [True, False], ids=["loss", "backward"])
def test_distill_error_flag_off_everything(loss_call):
    for p in (at(5, 16), at(9, 16), at(11), at(8)):
        refused(distill(loss_call, err=p), b"overlap")
    if loss_call:
        refused(distill(True, err=at(7, 8)), b"overlap")


def test_distill_backward_workspace_off_the_normaliser():
    refused(distill(False, ws=at(8)), b"overlap")


def test_lists_of_clients_without_weight_do_not_count():
    # the last check is the one that refuses: loss and lse are the same
    refused(distill(True, n=(1, 0), loss=at(2), lse=at(2)), b"loss and lse must not overlap")
    assert b"lists" not in fa.load().fedavg_last_error()


@pytest.mark.parametrize("i", [1, 2, 3, 4], ids=["x", "w", "bias", "residual"])
def test_forward_workspace_off_the_inputs(i):
    refused(forward(ws=at(i), wsb=1 << 20), b"workspace")


@pytest.mark.parametrize("i", [1, 2, 3, 4], ids=["dy", "x", "w", "preact"])
def test_backward_workspace_off_the_inputs(i):
    refused(backward(ws=at(i)), b"workspace")


def test_top_logits_workspace_off_the_logits():
    refused(topk(ws=at(1)), b"workspace")
