// Bit masks of draft trees from parent lists.
//
// Node i of a sequence names its parent, a node before it, or -1 for a root;
// it sees itself and its ancestors.  Bit j % 32 of word j / 32 of row i of the
// mask is set when node i sees node j, the form that the tree decode takes.
// One thread per (sequence, node) walks up the parents; a walk strictly
// descends, so it ends after at most i steps whatever the list holds (a parent
// outside [-1, i) sets a status bit and counts as -1).
#include <cuda_runtime.h>

#include "mla_internal.h"
#include "mla_sm103.cuh"

namespace mla {
namespace {

constexpr int kMaskThreads = 128;

__global__ void __launch_bounds__(kMaskThreads)
tree_mask_kernel(const int32_t *__restrict__ parents, int nodes, int s_q, uint32_t *__restrict__ mask, unsigned int *status) {
    sm103::griddep_wait();
    const int t = blockIdx.x * kMaskThreads + threadIdx.x;
    if (t >= nodes) return;
    const int i = t % s_q, words = (s_q + 31) / 32;
    const int32_t *up = parents + (t - i);
    uint32_t *row = mask + (size_t)t * words;
    // nodes come in descending order along a walk: one word is finished before the next begins
    int w = words - 1, j = i;
    uint32_t bits = 0;
    while (j >= 0) {
        while (w > (j >> 5)) {
            row[w--] = bits;
            bits = 0;
        }
        bits |= 1u << (j & 31);
        int next = up[j];
        if (next < -1 || next >= j) {
            atomicOr(status, MLA_DEVERR_SEQLEN);
            next = -1;
        }
        j = next;
    }
    while (w >= 0) {
        row[w--] = bits;
        bits = 0;
    }
}

}  // namespace

cudaError_t launch_tree_mask(const int32_t *parents, int batch, int s_q, uint32_t *mask, unsigned int *status,
                             cudaStream_t stream) {
    const int nodes = batch * s_q;
    return launch_after(tree_mask_kernel, dim3((unsigned)((nodes + kMaskThreads - 1) / kMaskThreads)), dim3(kMaskThreads), 0,
                        stream, parents, nodes, s_q, mask, status);
}

}  // namespace mla
