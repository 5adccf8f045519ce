// kv_select.cu -- which tokens of a cache stay: the first ones, the last ones, and of the
// others those with the largest weights.
//
// A sequence's weights are read once, as 32-bit keys in the order of the numbers (tokens
// that stay in any case above all, NaN below all), into the shared memory of a cluster of
// blocks, a run of tokens to a block.  The key of the budget-th token is found digit by
// digit (11, 11 and 10 bits): each pass counts the keys that share the digits found so far,
// the cluster adds its counts up in its first block (whole numbers: the order of the
// additions does not show), which finds the digit and tells the others.  Then every warp
// counts what it keeps, and after a sum over warps and blocks writes its tokens in
// ascending order; ties are taken from the lowest index on.
//
// Bound: latency (a call reads little: 64 sequences of up to 16384 tokens are 2 MB).
#include <algorithm>

#include "kv_attn_tile.cuh"

namespace kvr {

namespace {

constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32;
constexpr int kSelBins = 2048;
constexpr int kSelCluster = 8;   // most blocks of a sequence
constexpr int kSelSlice = 2048;  // fewest tokens that are worth a block
constexpr int kSelHeld = 49152;  // keys that a block holds; it reads others again

struct SelShared {
    uint32_t bins[kSelBins];
    uint32_t warp[2][kSelWarps];
    uint32_t above[kSelWarps];  // keys in the bins of later warps
    uint32_t digit, left;       // found by the cluster's first block
    uint32_t more[kSelCluster], same[kSelCluster]; // of every block, in each
};

// Order-preserving key of a weight.
__device__ __forceinline__ uint32_t weight_key(float w)
{
    const uint32_t b = __float_as_uint(w == 0.0f ? 0.0f : w); // -0 ties with 0
    if (w != w)
        return 0u;
    return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

__device__ __forceinline__ uint32_t remote_of(uint32_t smem, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem), "r"(rank));
    return r;
}

__device__ __forceinline__ void remote_add(uint32_t at, uint32_t v)
{
    asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

__device__ __forceinline__ void remote_st(uint32_t at, uint32_t v)
{
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

__global__ void __launch_bounds__(kSelThreads, 1) select_kernel(const __grid_constant__ SelectParams p)
{
    extern __shared__ uint32_t s_key[];
    __shared__ SelShared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int many = p.cluster, rank = (int)blockIdx.x % many, q = (int)blockIdx.x / many;
    const int len = __ldg(p.kv_len + q), budget = __ldg(p.budget + q);
    const bool fits =
        len >= 0 && len <= p.max_kv_len && budget >= 0 && min(len, budget) <= p.max_keep;
    if (tid == 0)
        write_block_status(p.header, fits ? kStatusOk : kStatusOutOfRange, blockIdx.x, gridDim.x);
    const int n = fits ? min(len, budget) : -1;
    if (rank == 0 && tid == 0)
        p.count[q] = n;
    if (n <= 0)
        return; // the same for the whole cluster
    const float *const weight = p.weights + q * p.weight_stride;
    int32_t *const keep = p.keep + q * p.keep_stride;
    float *const kept = p.kept ? p.kept + q * p.kept_stride : nullptr;
    const int sinks = min(p.sinks, len);
    const int tail = max(sinks, len - p.recent); // tokens from here on stay before others
    if (n == len || n <= sinks + len - tail) { // by place alone
        const int front = min(n, n == len ? n : sinks);
        for (int i = rank * kSelThreads + tid; i < n; i += many * kSelThreads) {
            const int at = i < front ? i : len - (n - i);
            keep[i] = at;
            if (kept)
                kept[i] = weight[at];
        }
        return;
    }
    // this block's tokens; a warp's are a run of whole 32s
    const int slice = (len + many - 1) / many, from = min(len, rank * slice);
    const int size = min(len, from + slice) - from;
    const int run = (size + kSelThreads - 1) / kSelThreads * 32;
    auto key_at = [&](int i) { // of the slice
        const int at = from + i;
        return at < sinks || at >= tail ? 0xFFFFFFFFu : weight_key(__ldg(weight + at));
    };
    auto key = [&](int i) { return i < kSelHeld ? s_key[i] : key_at(i); };
    for (int i = tid; i < min(size, kSelHeld); i += kSelThreads)
        s_key[i] = key_at(i);

    uint32_t prefix = 0, left = (uint32_t)n; // digits found; keys still wanted among those
    const uint32_t bins = smem_u32(sh.bins);
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
        for (int i = tid; i < kSelBins; i += kSelThreads)
            sh.bins[i] = 0;
        __syncthreads();
        for (int i = warp * 32 + lane; i - lane < size; i += kSelThreads) {
            const uint32_t k = i < size ? key(i) : 0u;
            const bool in = i < size && (pass == 0 || (k >> (shift + bits)) == prefix);
            const uint32_t who = __ballot_sync(0xFFFFFFFFu, in);
            if (!who)
                continue;
            // tokens that were never seen share a key: one addition for a warp of them
            const uint32_t bin = (k >> shift) & ((1u << bits) - 1u);
            const uint32_t lead = __shfl_sync(0xFFFFFFFFu, bin, __ffs((int)who) - 1);
            if (__all_sync(0xFFFFFFFFu, !in || bin == lead)) {
                if (lane == 0)
                    atomicAdd(&sh.bins[lead], (uint32_t)__popc(who));
            } else if (in) {
                atomicAdd(&sh.bins[bin], 1u);
            }
        }
        if (many > 1) {
            cluster_sync(); // the first block's own counts are in
            if (rank > 0)
                for (int i = tid; i < kSelBins; i += kSelThreads)
                    if (const uint32_t c = sh.bins[i])
                        remote_add(remote_of(bins + i * 4, 0), c);
            cluster_sync();
        } else {
            __syncthreads();
        }
        if (rank == 0) {
            // the bin in which the left-th largest key lies: a thread holds two bins
            const uint32_t c0 = sh.bins[2 * tid], c1 = sh.bins[2 * tid + 1];
            uint32_t sum = c0 + c1; // of this and the later lanes
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const uint32_t o = __shfl_down_sync(0xFFFFFFFFu, sum, d);
                if (lane + d < 32)
                    sum += o;
            }
            if (lane == 0)
                sh.warp[0][warp] = sum;
            __syncthreads();
            if (warp == 0) {
                uint32_t s = sh.warp[0][lane];
                const uint32_t mine = s;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const uint32_t o = __shfl_down_sync(0xFFFFFFFFu, s, d);
                    if (lane + d < 32)
                        s += o;
                }
                sh.above[lane] = s - mine;
            }
            __syncthreads();
            const uint32_t upto = sh.above[warp] + sum;  // keys from bin 2 tid on
            const uint32_t past = upto - c0 - c1;        // beyond this thread's bins
            if (past < left && left <= upto) {
                const bool high = left <= past + c1;
                const uint32_t digit = 2 * tid + (high ? 1 : 0);
                const uint32_t rest = left - past - (high ? 0 : c1);
                for (int r = 0; r < many; ++r) {
                    remote_st(remote_of(smem_u32(&sh.digit), r), digit);
                    remote_st(remote_of(smem_u32(&sh.left), r), rest);
                }
            }
        }
        if (many > 1)
            cluster_sync();
        else
            __syncthreads();
        prefix = pass == 0 ? sh.digit : prefix << bits | sh.digit;
        left = sh.left;
    }
    // keys above prefix stay, and the first `left` of those equal to it
    const int a = warp * run, b = min(size, a + run);
    uint32_t more = 0, same = 0;
    for (int i = a + lane; i < b; i += 32) {
        const uint32_t k = key(i);
        more += k > prefix;
        same += k == prefix;
    }
    more = __reduce_add_sync(0xFFFFFFFFu, more);
    same = __reduce_add_sync(0xFFFFFFFFu, same);
    if (lane == 0) {
        sh.warp[0][warp] = more;
        sh.warp[1][warp] = same;
    }
    __syncthreads();
    uint32_t before_more = 0, before_same = 0;
    {
        const uint32_t m = sh.warp[0][lane], s = sh.warp[1][lane];
        before_more = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? m : 0u);
        before_same = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? s : 0u);
        if (many > 1) {
            const uint32_t all_more = __reduce_add_sync(0xFFFFFFFFu, m);
            const uint32_t all_same = __reduce_add_sync(0xFFFFFFFFu, s);
            if (warp == 0 && lane < many) {
                remote_st(remote_of(smem_u32(&sh.more[rank]), lane), all_more);
                remote_st(remote_of(smem_u32(&sh.same[rank]), lane), all_same);
            }
        }
    }
    if (many > 1) {
        cluster_sync(); // no block reads another's memory after this
        for (int r = 0; r < rank; ++r) {
            before_more += sh.more[r];
            before_same += sh.same[r];
        }
    }
    for (int i = a + lane; i - lane < b; i += 32) {
        const uint32_t k = i < b ? key(i) : 0u;
        const uint32_t gt = __ballot_sync(0xFFFFFFFFu, i < b && k > prefix);
        const uint32_t eq = __ballot_sync(0xFFFFFFFFu, i < b && k == prefix);
        const uint32_t lower = (1u << lane) - 1u;
        const uint32_t e = before_same + __popc(eq & lower);
        if (((gt >> lane) & 1u) || (((eq >> lane) & 1u) && e < left)) {
            const uint32_t at = before_more + __popc(gt & lower) + min(e, left);
            keep[at] = from + i;
            if (kept)
                kept[at] = __ldg(weight + from + i);
        }
        before_more += __popc(gt);
        before_same += __popc(eq);
    }
}

} // namespace

int select_cluster(int32_t num_seqs, int32_t max_kv_len)
{
    int c = 1; // as many as keep the SMs busy, none with a short run
    while (c < kSelCluster && 2 * c * num_seqs <= kSms && max_kv_len >= 2 * c * kSelSlice)
        c *= 2;
    return c;
}

cudaError_t launch_select(const SelectParams &p, cudaStream_t stream)
{
    const int64_t slice = ((int64_t)p.max_kv_len + p.cluster - 1) / p.cluster;
    const int bytes = (int)std::min<int64_t>(slice, kSelHeld) * 4;
    cudaError_t e = allow_smem<select_kernel>(kSelHeld * 4);
    if (e != cudaSuccess)
        return e;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)p.cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(p.num_seqs * p.cluster));
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = (size_t)bytes;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, select_kernel, p);
}

} // namespace kvr
