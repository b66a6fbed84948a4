// afx_decode.hip -- the GPU restore of losslessly coded BF16 weights (gfx950).
//
// "Why Weight Offloading Slows Inference" (section "Three steps for each
// weight", Eq. (1)) names the unpack time t_unpack that every compressed
// weight pays before use; section "Lossless compression" entropy-codes the
// BF16 exponent field, so the unpack reconstructs each weight's exact bits.
// Here that unpack runs on the GPU after the compressed bytes reach device
// memory.
//
// Work decomposition (one launch per batch of up to 32 tensors):
//   * one workgroup of 16 wave64s fills a CU (4 waves per SIMD). The grid
//     is split among the batch's tensors by their chunk (4096-element)
//     counts (afx_split.h), so a workgroup serves about one tensor; within
//     a tensor the chunks go round its workgroups, so that all of them move
//     through each array together, in one narrow band;
//   * the waves of a workgroup claim its chunks one at a time from a counter
//     in LDS. A SIMD issues for its oldest waves first, so waves run at
//     different speeds; claiming keeps them finishing together;
//   * for every tensor it serves, the workgroup builds the 4096-entry decode
//     table (u16: symbol << 8 | length) of that tensor's canonical code in
//     LDS, from the 256 code lengths alone, and from it the pair table (u32:
//     both codes that start a 12-bit window when both fit in it);
//   * each wave restores one chunk at a time, software-pipelined: while chunk
//     i decodes, the code words and gap offsets of chunk i + 1 and the bit
//     bases of chunk i + 2 are in flight. The code words are staged in the
//     wave's own LDS slice; lane j then decodes groups j and j + 64 (32
//     symbols each, two independent dependency chains), two symbols per
//     32-bit window of the staged stream, mostly with one pair-table read;
//   * decoded exponent bytes go back to the wave's LDS slice in element order;
//     the wave re-reads them in store order, merges them with the
//     sign/mantissa bytes and writes 16-byte stores, 1 KB per instruction.
// There is no floating point and no matrix work: the kernel is bound by HBM
// bytes, and its first and last chunks by the serial table-lookup chain of
// each lane.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <vector>

#include "afx_device.h"

namespace afx {
namespace {

// Restored values go to the tensor's output in element order.
struct OutPlace {
    uint16_t *out;
    __device__ OutPlace(const TensorDesc &T, uint64_t e0) : out(T.out + e0) {}
    __device__ uint16_t *at(uint32_t i) const { return out + i; }
};

}  // namespace
}  // namespace afx

#include "afx_restore_body.h"

namespace afx {
namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int check_job(const afx_job &j) {
    int rc = check_info(j.info);
    if (rc != AFX_OK) return rc;
    if (!j.blob_dev || (!j.out_dev && j.info->n_elems)) return AFX_E_INVALID_ARG;
    if (j.out_bytes < j.info->decoded_bytes) return AFX_E_BUFFER_TOO_SMALL;
    if (!aligned16(j.blob_dev) || !aligned16(j.out_dev)) return AFX_E_MISALIGNED;
    if (j.info->n_elems) {
        const uintptr_t b0 = reinterpret_cast<uintptr_t>(j.blob_dev), b1 = b0 + j.info->blob_bytes;
        const uintptr_t o0 = reinterpret_cast<uintptr_t>(j.out_dev), o1 = o0 + j.info->decoded_bytes;
        if (o0 < b1 && b0 < o1) return AFX_E_INVALID_ARG;  // output overlaps the blob
    }
    return AFX_OK;
}

// The jobs of one call may run in one launch: no job's output may share a
// byte with another job's output or with any job's blob (check_job has
// compared each output with its own blob). Sorted by address, the outputs
// must be disjoint, and each blob must miss the output that starts last at
// or below its end (the outputs being disjoint, that is the only one that
// can reach into it). O(n log n): a whole model's tensors in one call.
// Returns -1 when host memory for the sort cannot be had (more than
// kStackRanges jobs only).
int outputs_overlap(const afx_job *jobs, size_t n) {
    struct Range {
        uintptr_t lo, hi;  // [lo, hi)
    };
    // the outputs' ranges: on the stack for up to kStackRanges jobs (a whole
    // model's tensors), on the heap beyond
    constexpr size_t kStackRanges = 1024;
    Range local[kStackRanges];
    std::vector<Range> heap;
    Range *outs = local;
    if (n > kStackRanges) {
        try {
            heap.resize(n);
        } catch (...) {
            return -1;
        }
        outs = heap.data();
    }
    size_t k = 0;
    for (size_t i = 0; i < n; ++i) {
        const uintptr_t o = reinterpret_cast<uintptr_t>(jobs[i].out_dev);
        if (jobs[i].info->decoded_bytes) outs[k++] = Range{o, o + jobs[i].info->decoded_bytes};
    }
    std::sort(outs, outs + k, [](const Range &a, const Range &b) { return a.lo < b.lo; });
    for (size_t i = 1; i < k; ++i)
        if (outs[i].lo < outs[i - 1].hi) return 1;
    for (size_t i = 0; i < n; ++i) {
        if (!jobs[i].info->n_elems) continue;
        const uintptr_t b0 = reinterpret_cast<uintptr_t>(jobs[i].blob_dev), b1 = b0 + jobs[i].info->blob_bytes;
        // the last output starting below the blob's end
        const Range *it = std::lower_bound(outs, outs + k, b1, [](const Range &r, uintptr_t v) { return r.lo < v; });
        if (it != outs && (it - 1)->hi > b0) return 1;
    }
    return 0;
}

// Enqueue one launch for up to AFX_MAX_JOBS_PER_LAUNCH already-checked jobs,
// on at most cap workgroups (cap >= 1).
int launch(const afx_job *jobs, size_t n_jobs, uint32_t cap, hipStream_t stream) {
    Batch batch;
    batch.n_tensors = 0;
    uint64_t chunks[AFX_MAX_JOBS_PER_LAUNCH];
    uint32_t lo[AFX_MAX_JOBS_PER_LAUNCH], hi[AFX_MAX_JOBS_PER_LAUNCH];
    uint32_t n_big = 0;
    // Tensors of fewer chunks than a workgroup has waves (a layer's norm
    // vectors) go last: together they are then a sliver of the grid's last
    // share, served by a workgroup of their own (each tensor a workgroup
    // serves costs it a table build), not added to one that also serves a
    // share of a large tensor.
    for (int pass = 0; pass < 2; ++pass) {
        for (size_t i = 0; i < n_jobs; ++i) {
            const uint64_t nc = jobs[i].info->n_chunks;
            if (nc == 0 || (pass == 0) != (nc >= kWavesPerBlock)) continue;
            chunks[batch.n_tensors] = nc;
            batch.t[batch.n_tensors++] = describe(jobs[i]);
            n_big += pass == 0 ? 1u : 0u;
        }
    }
    if (batch.n_tensors == 0) return AFX_OK;
    int max_blocks = 0;
    int rc = max_blocks_for_current_device(&max_blocks);
    if (rc != AFX_OK) return rc;
    max_blocks = (int)std::min<uint64_t>((uint64_t)max_blocks, cap);
    const uint32_t grid = split_grid(chunks, batch.n_tensors, n_big, (uint32_t)max_blocks, lo, hi);
    for (uint32_t t = 0; t < batch.n_tensors; ++t) {
        batch.t[t].blk_lo = lo[t];
        batch.t[t].blk_hi = hi[t];
    }
    // hipLaunchKernel reports this launch's own status (an error left pending
    // by an earlier, unrelated HIP call is not mistaken for it)
    void *args[] = {&batch};
    return hipLaunchKernel(reinterpret_cast<const void *>(&afx_decode_kernel), dim3((unsigned)grid), dim3(kThreads),
                           args, 0, stream) == hipSuccess
               ? AFX_OK
               : AFX_E_HIP;
}

// Every check of a batch call's jobs.
int check_batch(const afx_job *jobs, size_t n_jobs) {
    if (!jobs && n_jobs) return AFX_E_INVALID_ARG;
    for (size_t i = 0; i < n_jobs; ++i) {
        const int rc = check_job(jobs[i]);
        if (rc != AFX_OK) return rc;
    }
    const int ov = outputs_overlap(jobs, n_jobs);
    if (ov != 0) return ov < 0 ? AFX_E_HOST_MEMORY : AFX_E_INVALID_ARG;
    return AFX_OK;
}

// The launches of a checked batch call.
int decode_batch(const afx_job *jobs, size_t n_jobs, uint32_t cap, hipStream_t s) {
    for (size_t i = 0; i < n_jobs; i += AFX_MAX_JOBS_PER_LAUNCH) {
        const size_t k = std::min<size_t>(AFX_MAX_JOBS_PER_LAUNCH, n_jobs - i);
        const int rc = launch(jobs + i, k, cap, s);
        if (rc != AFX_OK) return rc;
    }
    return AFX_OK;
}

}  // namespace
}  // namespace afx

using namespace afx;

extern "C" {

int afx_decode_tensor(const afx_info *info, const void *blob_dev, void *out_dev, size_t out_bytes, void *stream) {
    const afx_job job{info, blob_dev, out_dev, out_bytes};
    int rc = check_job(job);
    if (rc != AFX_OK) return rc;
    hipStream_t s = static_cast<hipStream_t>(stream);
    rc = launch(&job, 1, UINT32_MAX, s);
    if (rc != AFX_OK) return rc;
    return hipStreamSynchronize(s) == hipSuccess ? AFX_OK : AFX_E_HIP;
}

int afx_decode_layer_async(const afx_job *jobs, size_t n_jobs, void *stream) {
    const int rc = check_batch(jobs, n_jobs);
    return rc != AFX_OK ? rc : decode_batch(jobs, n_jobs, UINT32_MAX, static_cast<hipStream_t>(stream));
}

int afx_decode_layer_grid_async(const afx_job *jobs, size_t n_jobs, uint32_t max_workgroups, void *stream) {
    if (max_workgroups == 0) return AFX_E_INVALID_ARG;
    const int rc = check_batch(jobs, n_jobs);
    return rc != AFX_OK ? rc : decode_batch(jobs, n_jobs, max_workgroups, static_cast<hipStream_t>(stream));
}

}  // extern "C"
