/*
 * ar.h -- C ABI of the GB300 virtual-rank allreduce library
 *         (libar_gb300.so).
 *
 * R "virtual ranks" are R separate buffers in the HBM of ONE GPU.  An
 * allreduce leaves, in every rank's output buffer, the element-wise sum of
 * all R input buffers:
 *
 *     out_r[i] = rne( ((float)in_0[i] + (float)in_1[i]) + ... + (float)in_{R-1}[i] )
 *
 * for every r in [0, R) and i in [0, count): fp32 additions in rank order
 * 0..R-1 (seeded with rank 0's value, no fused multiply-add), one final
 * round-to-nearest-even to the element type (bf16 or fp16; none for fp32).
 * Every variant below produces this result bit for bit; they differ only in
 * how the data moves.
 *
 * Where each operation comes from:
 *   - the input/output pointer tables mirror the broadcast table of output
 *     pointers of "optimize allreduce write mode by broadcast output ptr"
 *     (ROCm/aiter #1910, Motivation and Technical Details) and the device
 *     array of peer pointers passed as a kernel argument in "One shot all
 *     reduce Example" (pytorch-labs/helion #245, review discussion);
 *   - AR_ONESHOT_PULL is the one-shot allreduce of "One shot all reduce
 *     Example" (every rank reads all peers and reduces locally);
 *   - AR_ONESHOT_FANOUT is that one-shot read combined with the write mode of
 *     the aiter page (the reduced value is written straight into every
 *     rank's output through the output-pointer table);
 *   - AR_TWOPHASE is the two-stage allreduce of the aiter page without write
 *     mode (stage 1 reduces a shard into its owner's output, stage 2 copies
 *     it into the other ranks' outputs);
 *   - AR_ONESHOT_FANOUT_BULK is the same fan-out with every input tile
 *     brought into shared memory, and every result tile sent to the R
 *     outputs, by the bulk-copy (TMA) engine;
 *   - AR_FUSED_LL8_STAGED is the fused kernel below without write mode,
 *     otherwise the same kernel: each owner sends its reduced shard back as
 *     LL8 packets to every rank's result slot and every rank copies them
 *     into its output (the packet broadcast of the ARK page);
 *     AR_PACKET_3OP runs the three phases as three launches over the whole
 *     message (that page's send_packet -> recv_reduce_send_packet ->
 *     recv_packet decomposition).  Both exist to measure what write mode
 *     and fusion save;
 *   - AR_FUSED_LL8 is the single fused scatter -> reduce -> broadcast kernel
 *     synchronised by LL packet flags of "Add monolithic fused packet
 *     allreduce kernel and Model::all_reduce_packet API" (microsoft/ark #254,
 *     Changes), with the flag rotated on every call (that page's Known
 *     limitations leave Flag = 1 hardcoded), and the broadcast done in the
 *     aiter write mode.  Each CTA holds one warp group per virtual rank, so
 *     packet exchanges stay within a CTA and no CTA waits on another (the
 *     page's NumProcs >= NPeers limitation cannot arise); the kernel is
 *     pipelined over rounds so that its packets stay in L2.
 *
 * Threading: the operators that take no handle may be called from several host
 * threads at once.  A handle may be used from one host thread at a time.  Calls on
 * one handle must be ordered on one stream (one call in flight), because a
 * handle owns one packet scratch region and one epoch; use one handle per
 * concurrent stream.  (The one-shot region of "Add HIP-graph capture
 * coverage for the sharded-relay collectives" (meta-pytorch/torchcomms
 * #3850, region-lifetime commit) has the same precondition.)
 *
 * Launch overlap: the one-shot, two-phase, bulk fan-out, reduce-scatter and
 * all-gather kernels of a call that moves at most 16 MiB (two-phase: 8 MiB)
 * are launched with programmatic dependent launch, so they may be scheduled
 * while the previous kernel in the stream is still running; each waits for that kernel to
 * complete (and its writes to be visible) before touching global memory, so
 * results are those of plain stream order.  The environment variable
 * AR_PDL=0, read by ar_create, turns this off.  The two pipelined fused
 * kernels (AR_FUSED_LL8, AR_FUSED_LL8_STAGED) are launched this way at every
 * size unless AR_PDL=0 or AR_FUSED_PDL=0; the three-launch packet form never
 * is.  Such a kernel reads the two pointer tables (not the buffers they
 * point to) before that wait, so the table round trip overlaps the previous
 * kernel's tail.  Hence a precondition: the tables must not be written by
 * the kernel just before the call in the same stream if that kernel lets
 * its dependents start early (griddepcontrol.launch_dependents) before it
 * writes them.  Tables written by a copy, a memset, any kernel without such
 * a trigger, or an earlier call of this library (which never writes them)
 * are safe.
 *
 * Streams are passed as `void*` holding a cudaStream_t (NULL = the legacy
 * default stream), so that this header needs no CUDA header.
 */
#ifndef AR_GB300_H
#define AR_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define AR_MAX_RANKS 16        /* one-shot, two-phase, reduce-scatter, all-gather */
#define AR_MAX_PACKET_RANKS 8  /* the LL8 packet variants */

typedef struct ar_ctx* ar_handle_t;

typedef enum {
  AR_BF16 = 0, /* bfloat16, 2 bytes: fp32 accumulation, one round to nearest even */
  AR_FP16 = 1, /* IEEE binary16, 2 bytes: fp32 accumulation, one round to nearest even */
  AR_FP32 = 2  /* IEEE binary32, 4 bytes: fp32 accumulation, no final rounding */
} ar_dtype_t;

typedef enum {
  AR_OK = 0,
  AR_ERR_INVALID_ARG = 1, /* bad R, count, pointer, variant or handle */
  AR_ERR_UNSUPPORTED = 2, /* unknown dtype, a packet variant with R > 8, no sm_103 device,
                             or ar_allreduce_host under stream capture */
  AR_ERR_OOM = 3,         /* device allocation failed in ar_create */
  AR_ERR_CUDA = 4,        /* a CUDA runtime call failed (launch, copy, sync) */
  AR_ERR_TIMEOUT = 5      /* a packet wait inside the fused kernel gave up */
} ar_status_t;

typedef enum {
  AR_AUTO = 0,           /* per-size selector (measured table) picks one of the below */
  AR_ONESHOT_PULL = 1,   /* CTA (chunk, r) reads all R inputs, writes out_r only */
  AR_ONESHOT_FANOUT = 2, /* CTA reads all R inputs once, writes all R outputs */
  AR_TWOPHASE = 3,       /* launch 1: owner shards reduced; launch 2: shards copied out */
  AR_FUSED_LL8 = 4,      /* one persistent kernel: LL8 packet scatter, poll+reduce, write mode */
  AR_ONESHOT_FANOUT_BULK = 5, /* fan-out with tiles moved by bulk (TMA) copies through shared memory */
  AR_FUSED_LL8_STAGED = 6,    /* fused LL8 without write mode: result packets back to every rank */
  AR_PACKET_3OP = 7           /* the same three packet phases as three separate launches */
} ar_variant_t;

#define AR_NUM_VARIANTS 8

/* Static description of a handle (filled by ar_query). */
typedef struct {
  int R;                    /* virtual ranks */
  int dtype;                /* ar_dtype_t */
  size_t max_count;         /* largest count accepted by ar_allreduce */
  size_t scratch_bytes;     /* LL8 packet scratch owned by the handle (both regions) */
  int num_sms;              /* SMs of the device the handle lives on */
  int fused_max_ctas;       /* co-resident CTA limit used to size the fused grid */
  int fused_threads;        /* threads per CTA of the fused kernel (R warp groups) */
  int device;               /* CUDA device ordinal */
} ar_info_t;

/*
 * ar_create -- make a handle for R virtual ranks of up to `max_count`
 * elements each, on the current CUDA device.
 *   R          1 .. AR_MAX_RANKS (the LL8 packet variants need R <=
 *              AR_MAX_PACKET_RANKS; their scratch is allocated only then).
 *   max_count  >= 1; bounds `count` of later calls and sizes the scratch.
 *   dtype      AR_BF16, AR_FP16 or AR_FP32 (element type of every buffer).
 *   out        receives the handle (set to NULL on failure).
 * Allocates, on the current device, two packet scratch regions (scatter
 * packets and the staged variants' result packets), each
 * 32 * R * (R-1) * S bytes with S = ceil(ceil(max_count/G)/R) rounded up
 * to a multiple of 4, G = 8 elements per 16-byte group for bf16/fp16 and 4
 * for fp32 (about 4*(R-1)*max_count bytes for 2-byte types), zeroed here
 * so that no flag matches a live epoch, then written back from L2 to memory
 * (the fused kernel drops consumed packet lines from L2 without writing
 * them back, so they read back as these zeros or as older packets; the
 * write-back writes a temporary buffer of twice the L2 size, about 256 MB,
 * freed before ar_create returns, unless AR_FUSED_DISCARD=0); the fused
 * kernel's per-CTA packet rings (3 rounds of (R-1)*32 bytes per co-resident
 * thread, about 52 MB at R = 8, less for small max_count); and
 * a small state block (epoch, done counter, error word).  Synchronous; not
 * for stream capture.
 * Errors: AR_ERR_INVALID_ARG (R, max_count, out), AR_ERR_UNSUPPORTED (dtype,
 * or the current device is not compute capability 10.3), AR_ERR_OOM, AR_ERR_CUDA.
 * Source: the one-shot region of "Add HIP-graph capture coverage for the
 * sharded-relay collectives" (meta-pytorch/torchcomms #3850, the commit that
 * ties the region's lifetime to its communicator: created once with it, never
 * re-created while it lives, so the epoch never resets); scratch and peer
 * references set up once by Model::all_reduce_packet in "Add monolithic fused
 * packet allreduce kernel and Model::all_reduce_packet API" (microsoft/ark
 * #254, Changes).
 */
ar_status_t ar_create(int R, size_t max_count, int dtype, ar_handle_t* out);

/*
 * ar_allreduce -- out_r[i] = rne(sum over s in rank order of in_s[i])
 * for every r < R and i < count.
 *   h          handle from ar_create.
 *   d_in_tbl   DEVICE pointer to an array of R device pointers (8 bytes each,
 *              e.g. a CUDA int64 tensor of data_ptr()s); entry r is rank r's
 *              input buffer of `count` elements of the handle's dtype.
 *   d_out_tbl  DEVICE pointer to an array of R device pointers; entry r is
 *              rank r's output buffer of `count` elements.
 *   count      elements per rank, 0 .. max_count.  0 returns AR_OK, no launch.
 *   stream     cudaStream_t (as void*) the kernels are launched on.
 * The caller owns the buffers and both tables; they must stay valid and
 * unmodified until the call has completed on `stream`.  The kernels read the
 * tables on the device, so the host never dereferences them.
 * Aliasing: out_r may be exactly in_r (in place) for every variant, and any
 * output may alias any input exactly in AR_ONESHOT_FANOUT.  AR_ONESHOT_PULL
 * detects exact aliasing on the device and then writes every output from
 * one CTA per chunk.  Partially overlapping buffers are undefined.
 * Alignment: buffers 16-byte aligned take 16-byte vector loads and stores
 * (AR_ONESHOT_FANOUT: 32-byte ones for calls of at least 4 MiB per rank
 * when every pointer is 32-byte aligned and R <= 8); any misaligned pointer
 * switches that call to element-sized accesses (same result, slower),
 * decided on the device.
 * Allocates nothing, synchronises nothing, so it can be captured into a CUDA
 * graph; the fused kernel's epoch lives on the device and rotates on every
 * execution, including graph replays (by one per call, or, when the kernel
 * keeps its packets in per-CTA rings -- more than two L2 sizes of packets -- by
 * its number of rounds, one flag per round).
 * Errors: AR_ERR_INVALID_ARG (NULL handle or table, count > max_count),
 * AR_ERR_UNSUPPORTED (a packet variant forced with R > 8), AR_ERR_CUDA
 * (launch failure).  A packet wait that exceeds the spin limit
 * is reported later by ar_get_device_status (the outputs of that call are
 * then undefined).
 * Source: the allreduce with every rank's output pointer available inside
 * the kernel, broadcast once on the host in graph mode, of "optimize
 * allreduce write mode by broadcast output ptr" (ROCm/aiter #1910,
 * Motivation and Technical Details); the device array of peer pointers passed
 * as a kernel argument in "One shot all reduce Example" (pytorch-labs/helion
 * #245, review discussion); the fused kernel of microsoft/ark #254, Changes.
 */
ar_status_t ar_allreduce(ar_handle_t h, const void* const* d_in_tbl,
                         void* const* d_out_tbl, size_t count, void* stream);

/*
 * ar_reduce_scatter -- rank r keeps block r of the sum:
 *   out_r[j] = rne(sum over s in rank order of in_s[r*recvcount + j]),
 * j < recvcount.  Same numerics as ar_allreduce.  Each input holds
 * R*recvcount elements, each output recvcount elements; R*recvcount <=
 * max_count.  It is the one-shot push-reduce kernel of "Add HIP-graph
 * capture coverage for the sharded-relay collectives" (meta-pytorch/
 * torchcomms #3850) with a per-peer source stride of one block and an owner
 * offset of the rank's slot times one block; its allreduce case is the one
 * with a stride of zero.
 * ar_all_gather -- every output is the concatenation of all inputs in rank
 * order: out_r[s*sendcount + j] = in_s[j]; inputs hold sendcount elements,
 * outputs R*sendcount; R*sendcount <= max_count.
 * Both: device pointer tables as in ar_allreduce; outputs must not overlap
 * inputs; 16-byte vectors when every pointer is 16-byte aligned and the
 * block length is a multiple of the 16-byte group (8 elements of 2 bytes,
 * 4 of fp32), else element-sized accesses; one launch, no
 * allocation, no synchronisation.  Errors: AR_ERR_INVALID_ARG (NULL handle
 * or table, block too large), AR_ERR_CUDA (launch).  A block of 0 returns
 * AR_OK without a launch.
 */
ar_status_t ar_reduce_scatter(ar_handle_t h, const void* const* d_in_tbl,
                              void* const* d_out_tbl, size_t recvcount, void* stream);
ar_status_t ar_all_gather(ar_handle_t h, const void* const* d_in_tbl,
                          void* const* d_out_tbl, size_t sendcount, void* stream);

/* ar_destroy -- synchronise the device and free everything the handle owns.
 * NULL is accepted.  Returns AR_ERR_CUDA if a free failed.
 * Source: the region freed together with its communicator in the
 * region-lifetime commit of meta-pytorch/torchcomms #3850 (never freeing
 * leaked a region per communicator). */
ar_status_t ar_destroy(ar_handle_t h);

/* ar_set_variant -- force a variant for later calls on h (AR_AUTO restores
 * the selector).  AR_ERR_INVALID_ARG for an unknown value.
 * Source: the per-size choice between schedules at measured crossovers of
 * meta-pytorch/torchcomms #3850 (the commit re-measuring the relay/direct
 * crossovers), and the fixed block size that cost helion #245's one-shot
 * kernel at 1m (performance table note). */
ar_status_t ar_set_variant(ar_handle_t h, int variant);

/* ar_select -- the variant a call of `count` elements would run (the forced
 * one, or the selector's choice under AR_AUTO).  Host-only, no device work. */
ar_status_t ar_select(ar_handle_t h, size_t count, int* variant);

/* ar_set_launch -- override the CTA count and threads per CTA of a variant
 * (0 = automatic).  For AR_FUSED_LL8 and AR_FUSED_LL8_STAGED ctas is the
 * number of CTAs (each one clique of R warp groups), clamped to the
 * co-resident limit (and, in ring mode, to the packet rings' room), and
 * threads is rounded to R warp groups of a multiple of 32 threads each (at
 * least 32), narrowed where the kernel is compiled for fewer (AR_FUSED_LL8
 * for R <= 4 launches at most 256 threads); for the other variants ctas is
 * the grid (the grid-stride CTA
 * count; a multiple of R for the pull, two-phase and three-launch packet
 * kernels).  threads must be a multiple of 32 in [64, 512]
 * (the packet and fan-out kernels accept 128..512). */
ar_status_t ar_set_launch(ar_handle_t h, int variant, int ctas, int threads);

/* ar_set_spin_limit_ns -- the longest a fused-kernel packet wait may spin
 * before it gives up and sets the device error word (default 100 ms,
 * minimum 1000 ns).  Read by each later launch. */
ar_status_t ar_set_spin_limit_ns(ar_handle_t h, uint64_t ns);

/* ar_get_device_status -- wait (bounded: at most 60 s of polling) for
 * `stream` to drain, then read and clear the handle's device error word.
 * AR_OK, AR_ERR_TIMEOUT if some fused call since the last check gave up
 * waiting for packets, AR_ERR_CUDA if the stream did not drain or a copy
 * failed.
 * Source: the stream synchronise replaced by a bounded poll, so that a kernel
 * that never retires is reported instead of hanging, in the summary of
 * meta-pytorch/torchcomms #3850. */
ar_status_t ar_get_device_status(ar_handle_t h, void* stream);

/* ar_last_timeout -- details of the last AR_ERR_TIMEOUT that
 * ar_get_device_status returned on this handle (host-only, no device work):
 * *waiting_rank = the virtual rank whose packet wait gave up first,
 * *missing_rank = the lowest-numbered rank whose packets (scatter packets,
 * or result packets without write mode) it was still missing, *waits = how
 * many waits gave up before the others saw the call abandoned.  Waits for
 * result packets run twice the spin limit, so when a producer stores nothing
 * it is a wait for that producer's scatter packets that runs out first and
 * the producer that is named.  All -1 / 0
 * if no timeout has been reported.  AR_ERR_INVALID_ARG for a NULL argument.
 * Source: no counterpart on the pages; it names the peer that a bounded poll
 * (the summary of meta-pytorch/torchcomms #3850) gave up on, which a
 * multi-GPU caller would use to tell a dead peer from a slow one. */
ar_status_t ar_last_timeout(ar_handle_t h, int* waiting_rank, int* missing_rank,
                            uint32_t* waits);

/* ar_query -- fill *info. */
ar_status_t ar_query(ar_handle_t h, ar_info_t* info);

/* ar_status_string -- static, never NULL.
 * Source: the pages define no such function; it names the status codes
 * above, whose failure modes (a wait that never ends, reported rather than
 * hung on) come from the summary of meta-pytorch/torchcomms #3850. */
const char* ar_status_string(int status);

/* ar_variant_name -- static name of a variant ("auto", "oneshot_pull", ...),
 * "?" for an unknown value. */
const char* ar_variant_name(int variant);

/* ---- host-buffer path (end-to-end use from host memory) ----------------
 *
 * ar_reserve_host_staging -- allocate, once, R input and R output device
 * buffers of max_count elements plus their device pointer tables, used by
 * ar_allreduce_host.  Synchronous.  AR_ERR_OOM / AR_ERR_CUDA on failure.
 *
 * ar_allreduce_host -- h_in[r] / h_out[r] are HOST pointers (host arrays of
 * R host pointers).  When every buffer is page-locked (or device memory),
 * the kernel reads and writes the buffers where they are -- page-locked
 * host memory is device-addressable through unified addressing, over
 * NVLink-C2C on Grace-Blackwell -- so each input byte crosses to the device
 * once and each output byte back once, both directions concurrently; with
 * AR_AUTO this path runs AR_ONESHOT_FANOUT (one read and one write per
 * byte), otherwise the forced variant (AR_ONESHOT_FANOUT_BULK always
 * takes the staging path).  Otherwise (pageable memory) on
 * `stream`: one cudaMemcpyAsync per rank into the staging inputs, the
 * allreduce (same selection as ar_allreduce), one cudaMemcpyAsync per rank
 * back into h_out[r].  Returns after enqueueing; the caller synchronises
 * `stream` before reading h_out.  AR_ERR_INVALID_ARG if the staging was not
 * reserved or count > max_count.
 * Not capturable: a call on a stream that is being captured into a CUDA
 * graph returns AR_ERR_UNSUPPORTED and enqueues nothing (the device pointer
 * table is copied from memory that lives only for the duration of the call,
 * and pageable copies cannot be captured).  Capture ar_allreduce on device
 * buffers instead.
 */
ar_status_t ar_reserve_host_staging(ar_handle_t h);
ar_status_t ar_allreduce_host(ar_handle_t h, const void* const* h_in,
                              void* const* h_out, size_t count, void* stream);

/* ---- test hooks (faults made on the host side) --------------------------
 *
 * ar_debug_skip_producer -- for the NEXT call of a packet variant only
 * (AR_FUSED_LL8, AR_FUSED_LL8_STAGED, AR_PACKET_3OP), virtual rank `rank`
 * stores none of its scatter packets, so every owner's wait for that rank
 * runs out after the spin limit, the error word is set and ar_last_timeout
 * names `rank` as the missing one.  -1 clears.
 * No memory is touched out of bounds and no wait is unbounded.
 *
 * ar_debug_set_epoch / ar_debug_get_epoch -- synchronous write / read of
 * the device epoch (for testing the wrap from 2^32-1 to 1, which skips 0).
 * Setting it also zeroes every packet region (and writes the zeros back to
 * memory), so that no packet left from before the jump can match the new
 * epoch's flags (in normal use the epoch only moves forward one step per
 * call, and a stale match needs a full 2^32 wrap).
 */
ar_status_t ar_debug_skip_producer(ar_handle_t h, int rank);

/* ar_debug_check_guards -- synchronise the device, then check the guard
 * zones (4 KiB of a fixed byte value before and after each packet region the
 * handle owns: the scatter scratch, the result scratch and the rings), which
 * nothing in the library writes.  *intact = 1 if every guard byte still holds
 * its value, 0 if some kernel wrote outside a packet region.  AR_ERR_CUDA if
 * a copy fails, AR_ERR_INVALID_ARG for a NULL argument.  A stand-in for a
 * memory checker on the library's own buffers (output buffers belong to the
 * caller, who can surround them with guards of its own). */
ar_status_t ar_debug_check_guards(ar_handle_t h, int* intact);

/* ar_debug_delay_producer -- for every later AR_FUSED_LL8 or
 * AR_FUSED_LL8_STAGED call (until cleared with rank -1 or ns 0), the warps of
 * virtual rank `rank` wait `ns` nanoseconds of the device's global timer
 * before their first packet store,
 * so every owner polls for that rank's packets longer than the others'.
 * This is the skewed producer of "Add HIP-graph capture coverage for the
 * sharded-relay collectives" (meta-pytorch/torchcomms #3850, summary:
 * replays with some ranks delayed so that a stale flag or stale staging
 * fails deterministically), made on one GPU.  The value is taken at launch,
 * so a captured call keeps it on every replay.  The wait is bounded (ns <=
 * 10 ms, AR_ERR_INVALID_ARG above) and shorter than any spin limit a test
 * sets, so no wait runs out because of it. */
ar_status_t ar_debug_delay_producer(ar_handle_t h, int rank, uint64_t ns);
ar_status_t ar_debug_set_epoch(ar_handle_t h, uint32_t epoch);
ar_status_t ar_debug_get_epoch(ar_handle_t h, uint32_t* epoch);

/* ---- allocation-free entry point ----------------------------------------
 *
 * The pages have no counterpart to this call; it exists for callers of this
 * library that cannot allocate device memory themselves, so cannot use
 * ar_create: for example a plugin running inside a host framework whose
 * allocator has already reserved the device memory budget and forbids side
 * allocations, or a process that must not allocate once it has started
 * serving.
 *
 * ar_allreduce_fused_noalloc -- the AR_FUSED_LL8 allreduce of bf16 buffers
 * (R <= AR_MAX_PACKET_RANKS) without a handle.
 * Same arguments and result as ar_allreduce (R = rank count,
 * 1..AR_MAX_PACKET_RANKS; device pointer tables; count elements per rank;
 * stream), but the packet
 * scratch and the epoch/counter/error block live in fixed arrays inside the
 * library's device image (AR_NOALLOC_SCRATCH_BYTES of scratch plus 64 bytes),
 * which every GPU that loads the library holds until the process exits.  It
 * calls no cudaMalloc, cudaFree or other allocating routine.
 *   - The first call on each device sets that device up, synchronously:
 *     it looks up the arrays' device addresses, zeroes the scratch and
 *     starts the epoch at 1.  Make that first call before any stream capture.
 *   - count must be <= AR_NOALLOC_MAX_COUNT(R) (about 1.19 M elements for
 *     R = 8, 8.4 M for R = 2, no limit for R = 1); a larger count returns
 *     AR_ERR_INVALID_ARG and launches nothing.  count = 0 returns AR_OK.
 *   - Every call on a device shares the one array and the one epoch, which
 *     keep the last call's contents; the kernel needs nothing cleared between
 *     calls (stale packets carry older epochs, the done counter is left at 0
 *     by the call before).  Calls that overlap on the GPU (other streams, or
 *     other threads) race on the array and give wrong results: order them.
 *   - A packet wait that gives up (100 ms) is recorded in the device-side
 *     error word, which no entry point reads back for this call; that call's
 *     outputs are then undefined.
 * Errors: AR_ERR_INVALID_ARG (R < 1 or R > AR_MAX_PACKET_RANKS, NULL table,
 * count too large), AR_ERR_UNSUPPORTED (device ordinal >= 64), AR_ERR_CUDA
 * (set-up or launch).
 */
#define AR_NOALLOC_SCRATCH_BYTES ((size_t)32 << 20)
#define AR_NOALLOC_MAX_COUNT(R)                                                   \
  ((R) <= 1 ? (size_t)-1                                                          \
            : (AR_NOALLOC_SCRATCH_BYTES / ((size_t)32 * (size_t)(R) * (size_t)((R)-1))) * \
                  (size_t)8 * (size_t)(R))
ar_status_t ar_allreduce_fused_noalloc(int R, const void* const* d_in_tbl,
                                       void* const* d_out_tbl, size_t count, void* stream);

/* ---- feed-forward operators around the sum ------------------------------
 *
 * A tensor-parallel layer's feed-forward block stands on both sides of the
 * allreduce: before it every rank computes its shard of the gated
 * projections and its partial down projection, whose R partial results
 * ar_allreduce sums; after it come dropout and the residual.  The calls
 * below are those steps for ONE rank's buffers (R virtual ranks: R calls).
 * The pages have no counterpart to them.
 *
 * Matrices are row-major device arrays: element (i, j) of a matrix with
 * leading dimension ld is at [i * ld + j], ld >= its columns, in elements.
 * Any ld and any element-aligned base address is accepted.  The products read
 * rows that start on 16 bytes (base and ld) as they are.  Other rows they copy
 * into `scratch` first: device memory, 16-byte aligned, of at least the bytes
 * that the call's _scratch_bytes function gives for the same operands (0 where
 * all rows start on 16 bytes; scratch may then be NULL), owned by the caller
 * and free again when the call has completed.  With scratch NULL such operands
 * take a slower kernel.  (Forward products of up to AR_FEW_TOKENS tokens read
 * any rows as they are and use no scratch.)  All calls are
 * asynchronous on `stream`, allocate nothing, synchronise nothing, and can be
 * captured into a CUDA graph.  Outputs must not overlap inputs or one another
 * unless a call says so.
 */
#define AR_FEW_TOKENS 32

typedef enum {
  AR_ACT_SILU = 0,      /* v / (1 + exp(-v)) */
  AR_ACT_GELU_TANH = 1  /* v/2 (1 + tanh(sqrt(2/pi) (v + 0.044715 v^3))) */
} ar_activation_t;

typedef struct ar_ffn_ctx* ar_ffn_t;

/* ar_ffn_create -- a handle for one rank's gated feed-forward shard on the
 * current CUDA device.
 *   max_tokens  >= 1: bounds `tokens` of ar_ffn_backward and sizes its workspace
 *               (ar_ffn_forward needs none and takes any number of tokens).
 *   hidden      >= 1: columns of x and of the weights (K below).
 *   width       >= 1: rows of each weight matrix, this rank's part of the
 *               block's inner width (F below).
 *   dtype       AR_BF16 or AR_FP16; AR_FP32 is AR_ERR_UNSUPPORTED (the
 *               products run on 16-bit tensor-core operands).
 *   activation  ar_activation_t.
 *   train       non-zero: allocate the workspace of ar_ffn_backward (two
 *               max_tokens x width matrices of dtype, and at most 128 rows more); zero: allocate nothing,
 *               and ar_ffn_backward returns AR_ERR_UNSUPPORTED.
 * ar_ffn_backward calls on one handle share the workspace: order them on one
 * stream.  ar_ffn_forward calls share nothing.
 * Errors: AR_ERR_INVALID_ARG, AR_ERR_UNSUPPORTED (dtype, or the device is not
 * compute capability 10.3), AR_ERR_OOM, AR_ERR_CUDA. */
ar_status_t ar_ffn_create(size_t max_tokens, size_t hidden, size_t width, int dtype,
                          int activation, int train, ar_ffn_t* out);

/* ar_ffn_destroy -- synchronise the device and free the handle.  NULL is
 * accepted.  Not while a stream is being captured, nor while a graph that holds
 * an ar_ffn_backward of the handle may still be launched: the graph keeps the
 * workspace's address. */
ar_status_t ar_ffn_destroy(ar_ffn_t h);

/* ar_ffn_forward -- out = act(x Wgate^T) * (x Wup^T), in one kernel.
 *   x             [tokens, hidden], leading dimension ldx
 *   w_gate, w_up  [width, hidden], both with leading dimension ldw
 *   out           [tokens, width], leading dimension ldo
 *   gate, up      NULL, or [tokens, width] with ldo: receive the two products
 *                 before the activation, rounded to dtype, which
 *                 ar_ffn_backward takes.  Both or neither.
 * Sums are held in fp32; the activation and the product are taken in fp32
 * from the unrounded sums; each output is rounded once, to nearest even.
 * tokens = 0 returns AR_OK without a launch.  Errors: AR_ERR_INVALID_ARG
 * (NULL, ld too small, an odd address, scratch too small), AR_ERR_CUDA. */
ar_status_t ar_ffn_forward(ar_ffn_t h, const void* x, size_t ldx, const void* w_gate,
                           const void* w_up, size_t ldw, void* out, void* gate, void* up,
                           size_t ldo, size_t tokens, void* scratch, size_t scratch_bytes,
                           void* stream);

/* ar_ffn_scratch_bytes -- bytes of scratch with which ar_ffn_forward and
 * ar_ffn_backward can lay these operands out (see above); 0 for a NULL handle.
 * Host-only. */
size_t ar_ffn_scratch_bytes(ar_ffn_t h, const void* x, size_t ldx, const void* w_gate,
                            const void* w_up, size_t ldw, size_t tokens);

/* ar_ffn_backward -- the gradients of ar_ffn_forward:
 *   dgate = dout * up * act'(gate),  dup = dout * act(gate)
 *   dx      = dgate Wgate + dup Wup      [tokens, hidden], leading dimension lddx
 *   dw_gate = dgate^T x,  dw_up = dup^T x   [width, hidden] each, lddw
 *   gate, up, dout   [tokens, width], all with leading dimension ldo
 *   dx           NULL: not computed
 *   dw_gate, dw_up   both NULL: not computed
 * Sums in fp32, outputs rounded once.  dgate and dup are rounded to dtype
 * between the two steps, since they are operands of 16-bit tensor-core
 * products; for at most 64 tokens they are kept as the sum of two numbers of
 * dtype (where rows start on 16 bytes, or scratch is given).  So in AR_FP16 a
 * value of them below 2^-25 counts as 0, and one above 65504 as infinite: scale
 * the loss, as for any gradients held in that type.  The gradients are written,
 * not added to what the outputs held.
 * tokens = 0 writes zeros to dw_gate and dw_up.
 * Errors: AR_ERR_INVALID_ARG (also tokens > max_tokens), AR_ERR_UNSUPPORTED
 * (handle made with train = 0), AR_ERR_CUDA. */
ar_status_t ar_ffn_backward(ar_ffn_t h, const void* x, size_t ldx, const void* w_gate,
                            const void* w_up, size_t ldw, const void* gate, const void* up,
                            const void* dout, size_t ldo, void* dx, size_t lddx, void* dw_gate,
                            void* dw_up, size_t lddw, size_t tokens, void* scratch,
                            size_t scratch_bytes, void* stream);

/* ar_dropout -- out = residual + (keep ? x / (1 - p) : 0).
 *   x, residual, out  [rows, cols] of dtype (AR_BF16, AR_FP16, AR_FP32);
 *             residual may be NULL (taken as 0); out may be exactly x or
 *             residual (same address and leading dimension).
 *   p         in [0, 1]: keep where draw >= rint(p 2^32); p = 1 drops all.
 *   seed, sequence, offset   element (i, j) draws word n mod 4 of
 *             Philox4x32-10 with key `seed` on the 128-bit counter
 *             {n / 4, sequence}, n = offset + i * cols + j.  Use a sequence
 *             for each layer and step; offset is the place of a block (a
 *             rank's part of a reduce-scatter) in the whole tensor.
 * The mask depends on (seed, sequence, n) alone and is never stored: ranks
 * with equal arguments draw equal masks, and ar_dropout_backward (dx = keep ?
 * dy / (1 - p) : 0; the residual's gradient is dy) draws it again.
 * Multiplied by 1 / (1 - p) and added in fp32 (one fused step), rounded once to dtype.  A
 * dropped element counts as 0 whatever it holds, infinities and NaN included.
 * Errors: AR_ERR_INVALID_ARG (NULL x or out, ld < cols, p outside [0, 1] or
 * NaN, offset + rows * cols past 2^64), AR_ERR_UNSUPPORTED (dtype). */
ar_status_t ar_dropout(const void* x, size_t ldx, const void* residual, size_t ldr, void* out,
                       size_t ldo, size_t rows, size_t cols, int dtype, double p, uint64_t seed,
                       uint64_t sequence, uint64_t offset, void* stream);
ar_status_t ar_dropout_backward(const void* dy, size_t lddy, void* dx, size_t lddx, size_t rows,
                                size_t cols, int dtype, double p, uint64_t seed,
                                uint64_t sequence, uint64_t offset, void* stream);

/* ar_quantize_rows -- 8-bit integers and one scale for each row (token):
 *   scale[i] = max_j |x[i, j]| / 127,  q[i, j] = rint(x[i, j] / scale[i])
 * with IEEE fp32 divisions and ties to even; q is in [-127, 127].  A row of
 * zeros gets scale 0 and zeros.  A row that holds an infinity or a NaN gets
 * that as its scale, and zeros, so that its products come out as NaN.
 *   x  [rows, cols] of dtype (AR_BF16, AR_FP16, AR_FP32);  q  [rows, cols];
 *   scale  rows floats.  rows = 0 returns AR_OK without a launch. */
ar_status_t ar_quantize_rows(const void* x, size_t ldx, int8_t* q, size_t ldq, float* scale,
                             size_t rows, size_t cols, int dtype, void* stream);

/* ar_linear_i8 -- y[m, n] = x_scale[m] * w_scale[n] * sum_k x[m, k] w[n, k].
 *   x  [tokens, in] int8, w  [out, in] int8 (any value, -128 included),
 *   x_scale  one float a token, w_scale  one float an output channel,
 *   y  [tokens, out] of dtype AR_BF16 or AR_FP16, leading dimension ldy.
 * Products are exact and sums are held in fp32: exact while partial sums stay
 * within 2^24 (always for in <= 1024).  Beyond, each addition may round or
 * truncate to 24 bits: the sum is within `in` times 2^-23 of the sum of the
 * products' absolute values.  The sum is multiplied by x_scale, then by w_scale,
 * and rounded once.
 * tokens = 0 returns AR_OK without a launch.
 * Errors: AR_ERR_INVALID_ARG, AR_ERR_UNSUPPORTED (dtype AR_FP32), AR_ERR_CUDA. */
ar_status_t ar_linear_i8(const int8_t* x, size_t ldx, const float* x_scale, const int8_t* w,
                         size_t ldw, const float* w_scale, void* y, size_t ldy, size_t tokens,
                         size_t in, size_t out, int dtype, void* scratch, size_t scratch_bytes,
                         void* stream);

/* ar_linear_i8_scratch_bytes -- as ar_ffn_scratch_bytes.  Host-only. */
size_t ar_linear_i8_scratch_bytes(const int8_t* x, size_t ldx, const int8_t* w, size_t ldw,
                                  size_t tokens, size_t in, size_t out);

/* ---- norms and the residual after the sum --------------------------------
 *
 * What a layer does with the sum before its next block reads it, in one pass
 * over the rows.  With N(v) = (v - mu) / sqrt(mean((v - mu)^2) + eps), mu the
 * row's mean (AR_NORM_LAYER) or 0 (AR_NORM_RMS):
 *   z = N(x) * (weight_offset + after_weight) + after_bias   the norm after a block
 *   r = residual_scale * residual + gate * z                 the residual stream
 *   y = N(r) * (weight_offset + weight) + bias               the norm before the next one
 * The pages have no counterpart to these calls.
 */
typedef enum { AR_NORM_RMS = 0, AR_NORM_LAYER = 1 } ar_norm_kind_t;

typedef struct {
  int kind;   /* ar_norm_kind_t */
  int dtype;  /* AR_BF16, AR_FP16 or AR_FP32, of every array of the call */
  size_t rows, cols;
  size_t gate_rows;  /* rows of the gate matrix, a divisor of rows: gate row g is of the
                        rows / gate_rows rows from g * rows / gate_rows on (1: a gate for
                        each column, rows: for each row, between them for each sequence);
                        0: no gate */
  double eps, residual_scale, weight_offset;
} ar_norm_t;

/* ar_residual_norm --
 *   x             [rows, cols], leading dimension ldx: the block's output
 *   residual      NULL (taken as 0), or [rows, cols]
 *   gate          [gate_rows, cols]; NULL where gate_rows is 0 (taken as 1)
 *   after_weight  NULL: z = x; else cols values.  after_bias: NULL (0) or cols
 *                 values; only with after_weight
 *   weight        NULL: no y; else cols values.  bias likewise
 *   r, y          [rows, cols]; r may be NULL (not wanted), y is NULL where weight is
 * Means, sums and products are fp32, the mean square being taken of the
 * differences from the mean; y is made from the unrounded r; each output is rounded once.
 * A row's values are its own: an infinity or NaN stays in its row.  Squares
 * are fp32: those that overflow (values from 10^19 on, in AR_FP32 and AR_BF16) make the
 * row's norm 0 or NaN, and a row whose squares all vanish is scaled by 1 / sqrt(eps).
 * r or y may be exactly x or residual (same address and leading dimension), not both the
 * same one; otherwise outputs overlap nothing.  rows = 0 returns AR_OK without a launch.
 * Errors: AR_ERR_INVALID_ARG (a NULL that is needed, ld < cols, an odd address, r = y,
 * cols = 0, gate_rows that does not divide rows, eps negative or not finite, neither weight nor
 * after_weight), AR_ERR_UNSUPPORTED (dtype, kind), AR_ERR_CUDA. */
ar_status_t ar_residual_norm(const ar_norm_t* n, const void* x, size_t ldx, const void* residual,
                             size_t ldres, const void* gate, size_t ldg, const void* after_weight,
                             const void* after_bias, const void* weight, const void* bias, void* r,
                             size_t ldr, void* y, size_t ldy, void* stream);

/* ar_residual_norm_backward -- the gradients, given dy and dr, those of y and r:
 *   g = dr + (gradient of N(r) (weight_offset + weight) + bias with respect to r, at dy)
 *   dresidual = residual_scale * g,   dgate = sum of g * z over a gate row's rows
 *   dz = gate * g,                    dx = gradient of z with respect to x, at dz
 *   dweight = sum over rows of dy * N(r),  dbias = sum of dy
 *   dafter_weight = sum over rows of dz * N(x),  dafter_bias = sum of dz
 *   dy   [rows, cols], NULL where weight is
 *   dr   [rows, cols], or NULL (taken as 0)
 *   x    the forward pass's; may be NULL where there is neither after_weight nor gate
 *   r    the forward pass's (its rounded output; x where nothing was added); may be
 *        NULL where weight is
 *   dx, dresidual, dgate, dweight, dbias, dafter_weight, dafter_bias
 *        NULL: not computed.  dgate has the leading dimension lddg.
 * Statistics are taken again from x and r; sums are fp32, in an order that
 * depends on the sizes, the device, which arrays are given and whether those that
 * are read or written start their rows on 16 bytes, and on nothing else: a call
 * repeated gives the same bits; outputs are rounded once and written, not added to.
 *   scratch  device memory on 16 bytes, of ar_residual_norm_scratch_bytes(rows,
 *            cols, how many of dgate, dweight, dbias, dafter_weight and
 *            dafter_bias are not NULL) bytes; NULL where that is 0
 * Outputs overlap neither inputs nor one another.
 * rows = 0 writes zeros to the gradients of the vectors. */
ar_status_t ar_residual_norm_backward(const ar_norm_t* n, const void* dy, size_t lddy, const void* dr,
                                      size_t lddr, const void* x, size_t ldx, const void* r, size_t ldr,
                                      const void* gate, size_t ldg, const void* after_weight,
                                      const void* after_bias, const void* weight, void* dx, size_t lddx,
                                      void* dresidual, size_t lddres, void* dgate, size_t lddg,
                                      void* dweight, void* dbias, void* dafter_weight,
                                      void* dafter_bias, void* scratch, size_t scratch_bytes,
                                      void* stream);

/* ar_residual_norm_scratch_bytes -- see ar_residual_norm_backward.  Host-only. */
size_t ar_residual_norm_scratch_bytes(size_t rows, size_t cols, int vectors);

/* ---- products with 4-bit weights ------------------------------------------
 *
 *   y[m, n] = sum_k x[m, k] * scale[n, k / group] * (q[n, k] - zero[n, k / group])
 * with q and zero whole numbers in 0 .. 15 (zero is 8 where there are none), a
 * scale of the activations' type for each channel and group of k, for a few
 * tokens in serving.  The weights are laid out once, when they are loaded: by
 * ar_pack_i4 from whole numbers a row, or by ar_quantize_i4 from a matrix.  The
 * pages have no counterpart to them.
 *
 * group is 32, 64 or 128; the last group of a row may be short.  The laid-out
 * arrays are device memory on 16 bytes that the caller owns: `data` and `scale`, and
 * `zero` where there are zero points, of the sizes that ar_i4_sizes gives.
 * Their order is the library's own.
 */
/* ar_i4_sizes -- *data_bytes, and *scales: how many scales (16 bits each) and how many zero
 * points (a byte each) the layout of `out` channels of `in` weights holds.  Host-only.
 * Errors: AR_ERR_INVALID_ARG (a size of 0 or above 2^30, another group, NULL). */
ar_status_t ar_i4_sizes(size_t out, size_t in, int group, size_t* data_bytes, size_t* scales);

/* ar_pack_i4 -- lays out
 *   q      [out, in] bytes, of which the low four bits count; leading dimension ldq
 *   scale  [out, ceil(in / group)], 16 bits each; lds
 *   zero   NULL, or like scale, a byte each, of which the low four bits count; ldz
 * into data, packed_scale and packed_zero (NULL where zero is).  Asynchronous. */
ar_status_t ar_pack_i4(const uint8_t* q, size_t ldq, const void* scale, size_t lds, const uint8_t* zero,
                       size_t ldz, size_t out, size_t in, int group, void* data, void* packed_scale,
                       void* packed_zero, void* stream);

/* ar_quantize_i4 -- lays out w [out, in] of dtype (AR_BF16, AR_FP16), each group by itself:
 *   without zero points  scale = max |w| / 7,  q = rint(w / scale) + 8 in 1 .. 15
 *   with zero points     scale = max(w, 0) / 15 - min(w, 0) / 15,
 *                        zero = rint(-min / scale),  q = rint(w / scale) + zero in 0 .. 15
 * in IEEE fp32, the scale rounded to dtype before it divides, results past either end
 * taken as that end.  A group of zeros has scale 0; one that holds an
 * infinity or a NaN has scale NaN.
 *   packed_zero  NULL: without zero points
 *   scratch      ar_quantize_i4_scratch_bytes of device memory on 16 bytes, free
 *                again when the call has completed */
ar_status_t ar_quantize_i4(const void* w, size_t ldw, size_t out, size_t in, int group, int dtype,
                           void* data, void* packed_scale, void* packed_zero, void* scratch,
                           size_t scratch_bytes, void* stream);
size_t ar_quantize_i4_scratch_bytes(size_t out, size_t in, int group);

/* ar_dequantize_i4 -- w[n, k] = scale * (q - zero), multiplied in fp32 and
 * rounded once to dtype: [out, in], leading dimension ldw (for a product of many tokens). */
ar_status_t ar_dequantize_i4(const void* data, const void* packed_scale, const void* packed_zero,
                             size_t out, size_t in, int group, int dtype, void* w, size_t ldw,
                             void* stream);

/* ar_linear_i4 -- the product above.
 *   x  [tokens, in] of dtype AR_BF16 or AR_FP16 (that of the scales), ldx
 *   y  [tokens, out] of dtype, ldy
 *   packed_zero  NULL: every zero is 8
 * q - zero is exact; a group's products are summed in fp32, multiplied by its
 * scale in fp32 and added; y is rounded once.  The weights are read once for
 * every AR_FEW_TOKENS tokens; tokens is at most 32 * 65535.
 * tokens = 0 returns AR_OK without a launch.  Asynchronous; needs no scratch.
 * Errors: AR_ERR_INVALID_ARG, AR_ERR_UNSUPPORTED (dtype), AR_ERR_CUDA. */
ar_status_t ar_linear_i4(const void* x, size_t ldx, const void* data, const void* packed_scale,
                         const void* packed_zero, void* y, size_t ldy, size_t tokens, size_t in,
                         size_t out, int group, int dtype, void* stream);

/* ---- a layer of gated experts for a few tokens ----------------------------
 *
 * A mixture-of-experts layer in serving: every token is sent to its top_k
 * experts, each a gated feed-forward block as above with a down projection, and
 * their outputs are summed by weight.  A rank may hold a part of the experts (or
 * of every expert's inner width); the ranks' partial outputs are what
 * ar_allreduce sums.  The pages have no counterpart to it.
 */
#define AR_MAX_EXPERTS 1024
#define AR_MAX_TOP_K 16

typedef struct {
  int dtype;         /* AR_BF16 or AR_FP16, of x, the weights and out */
  int logits_dtype;  /* AR_BF16, AR_FP16 or AR_FP32 */
  int activation;    /* ar_activation_t */
  int experts;       /* of the whole layer: columns of the logits, 1 .. AR_MAX_EXPERTS */
  int first_expert;  /* this rank holds experts first_expert .. */
  int local_experts; /* .. first_expert + local_experts - 1 */
  int top_k;         /* 1 .. the smaller of experts and AR_MAX_TOP_K */
  int normalize;     /* non-zero: a token's weights are made to sum to 1 */
  size_t hidden;     /* columns of x and of out (K), at most 2^22 */
  size_t width;      /* rows of an expert's gate and up projections (F), at most 2^22;
                        local_experts * hidden * width below 2^40 */
} ar_moe_t;

/* ar_moe_ffn --
 *   x              [tokens, hidden], leading dimension ldx
 *   logits         [tokens, experts], ldl: the router's
 *   w_gate, w_up   [local_experts, width, hidden]: rows ldw, experts esw elements apart
 *   w_down         [local_experts, hidden, width]: ldd, esd
 *   out            [tokens, hidden], ldo
 *   expert, weight NULL, or [tokens, top_k] without gaps: receive the routing
 * A token's experts are those of its top_k highest logits, the highest first
 * and equal ones by the lowest index; weight j is exp(logit_j) over the sum of
 * all experts' exp, or (normalize) of the chosen ones'.  An expert whose logit is
 * -infinity is never chosen: where fewer remain, expert is -1 and weight 0.  A
 * row with a NaN or +infinity has NaN weights.  With e = expert[t, j]:
 *   h   = act(x[t] Wgate_e^T) * (x[t] Wup_e^T)
 *   out[t] = sum over the j whose e this rank holds of weight[t, j] * (h Wdown_e^T)
 * and zeros where it holds none.  Sums, the activation and the weighting are fp32, out is rounded
 * once.  Between the two products h is held in dtype: as the sum of two numbers where scratch has
 * ar_moe_two_part_scratch_bytes, whose error is below that of out's rounding, or else rounded to
 * one, which makes the result's error 1.4 times that of its own rounding.  In AR_FP16 an |h| of
 * 65,520 or more is an infinity either way.  Each matrix of an expert with tokens is read
 * once for every AR_FEW_TOKENS tokens (more are taken in runs of that many).
 *   scratch  device memory on 16 bytes, at least ar_moe_scratch_bytes of it, not shared
 *            with a call that may run at the same time
 * tokens = 0 returns AR_OK without a launch.  Asynchronous on `stream`; out
 * overlaps no input.  Errors: AR_ERR_INVALID_ARG, AR_ERR_UNSUPPORTED (a dtype),
 * AR_ERR_CUDA. */
ar_status_t ar_moe_ffn(const ar_moe_t* m, const void* x, size_t ldx, const void* logits, size_t ldl,
                       const void* w_gate, const void* w_up, size_t ldw, size_t esw,
                       const void* w_down, size_t ldd, size_t esd, void* out, size_t ldo,
                       int32_t* expert, float* weight, size_t tokens, void* scratch,
                       size_t scratch_bytes, void* stream);

/* ar_moe_scratch_bytes, ar_moe_two_part_scratch_bytes -- see ar_moe_ffn; 0 for what it refuses.
 * Host-only. */
size_t ar_moe_scratch_bytes(const ar_moe_t* m, size_t tokens);
size_t ar_moe_two_part_scratch_bytes(const ar_moe_t* m, size_t tokens);

/* ar_ops_get_device_status -- wait for `stream` to drain, then read and clear
 * the feed-forward operators' error word on the current device: AR_ERR_TIMEOUT
 * if a wait inside one of their tensor-core kernels gave up (two seconds; such
 * a call's outputs are undefined), AR_ERR_CUDA if the stream did not drain.
 * No wait can run out in a working call: each is for a copy or a matrix
 * instruction that the same CTA, or its pair, has issued.  Not for stream
 * capture. */
ar_status_t ar_ops_get_device_status(void* stream);

#ifdef __cplusplus
}
#endif

#endif /* AR_GB300_H */
