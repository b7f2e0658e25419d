/*
 * logmel.h -- C ABI of liblogmel.so, the GB300 (sm_103a) log-mel front end.
 *
 * Two operations (and, in sections 4 to 6, what turns their features into
 * text: linear layers, an 8-bit key/value cache with its attention, and beam
 * search; in sections 7 to 9, the rest of such a model's layers: layer norm and
 * gated linear layers with their gradients, and weights in 4 bits):
 *
 *  1. lm_log_mel_from_stft: Whisper's log-mel spectrogram from a complex
 *     STFT, as defined by the KBench task spec "audio_mel_spectrogram_fused.py"
 *     (its reference function and the per-clip definition in its spec text):
 *         mag[b,f,k]      = re^2 + im^2                      (power)
 *         mel[b,f,n]      = sum_k mag[b,f,k] * mel_filters[n,k]
 *         log_spec[b,f,n] = log10(max(mel[b,f,n], 1e-10))
 *         hi[b]           = max over (f, n) of log_spec[b,f,n]  (per clip)
 *         out[b,f,n]      = (max(log_spec[b,f,n], hi[b] - 8) + 4) / 4
 *     All arithmetic is f32 (the spec's precision section rules out bf16,
 *     fp16 and fp8 anywhere on this path).
 *
 *  2. lm_mel_spectrogram: waveform -> mel spectrogram, the torchaudio-style
 *     MelSpectrogram described on the "flashmel" PyPI page (usage section and
 *     argument list): framing with center padding, periodic Hann window,
 *     one-sided real FFT, |X|^power, triangular mel filterbank (HTK or Slaney
 *     scale), f32 or int16 input (int16 scaled by 1/32768), f32 or f16
 *     output, laid out [B, n_mels, n_frames].  Optionally followed by the same
 *     log10 / per-clip clamp / rescale as operation 1.
 *
 * Conventions for every entry point:
 *  - Pointers named as device pointers must point to memory of the current
 *    CUDA device; the caller owns all buffers.  Inputs are read-only.
 *  - Work is enqueued asynchronously on `stream` (NULL = legacy default
 *    stream); results are ready once the stream reaches that point.
 *  - Nothing is allocated on the compute path: scratch comes from the
 *    caller's `workspace`, sized by the matching *_workspace_size call.
 *  - Errors are returned as lm_status, never by aborting or trapping.
 *    Argument errors are detected on the host before anything is enqueued.
 *    LM_ERR_CUDA means a CUDA runtime call failed; lm_last_cuda_error()
 *    returns its code (per host thread).
 *  - Kernels bound every wait they perform.  A wait that runs out (which
 *    correct use never triggers) sets a device error word in the workspace
 *    instead of hanging; lm_workspace_error() reads it.
 */
#ifndef LOGMEL_H_
#define LOGMEL_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t / CUstream. */
typedef struct CUstream_st *lm_stream_t;

typedef enum lm_status {
  LM_OK = 0,
  LM_ERR_INVALID_ARG = 1,   /* null pointer, negative or inconsistent size */
  LM_ERR_UNSUPPORTED = 2,   /* a valid request this library does not implement */
  LM_ERR_MISALIGNED = 3,    /* a pointer lacks the stated alignment */
  LM_ERR_CUDA = 4,          /* a CUDA runtime call failed, see lm_last_cuda_error */
  LM_ERR_OUT_OF_MEMORY = 5, /* plan creation could not allocate its tables */
  LM_ERR_DEVICE_FAULT = 6,  /* a kernel reported a bounded wait that ran out */
  LM_ERR_WORKSPACE = 7      /* workspace null or smaller than required */
} lm_status;

typedef enum lm_dtype { LM_F32 = 0, LM_I16 = 1, LM_F16 = 2, LM_BF16 = 3 } lm_dtype;

typedef enum lm_pad_mode {
  LM_PAD_REFLECT = 0,   /* mirror about the edge sample, edge not repeated */
  LM_PAD_CONSTANT = 1,  /* zeros */
  LM_PAD_REPLICATE = 2, /* repeat the edge sample */
  LM_PAD_CIRCULAR = 3   /* wrap around */
} lm_pad_mode;

typedef enum lm_mel_scale { LM_MEL_HTK = 0, LM_MEL_SLANEY = 1 } lm_mel_scale;

/* Human-readable name of a status code.  Never NULL. */
const char *lm_status_string(int status);

/* The cudaError_t of the last failed CUDA call made by this host thread
 * inside the library (0 if none). */
int lm_last_cuda_error(void);

/* Library version as major * 10000 + minor * 100 + patch. */
int lm_version(void);

/* ------------------------------------------------------------------------ */
/* 1. log-mel from a complex STFT                                           */
/* ------------------------------------------------------------------------ */

/* Bytes of device workspace lm_log_mel_from_stft needs for this shape
 * (a header, one u32 per clip and one u32 per tile of frames).  Host-only. */
lm_status lm_log_mel_from_stft_workspace_size(int64_t B, int64_t F, int32_t NF, int32_t NM,
                                              size_t *bytes);

/*
 * Whisper log-mel from a complex STFT (KBench "audio_mel_spectrogram_fused"
 * spec: reference function, per-clip definition and I/O contract).
 *
 *   stft        device, [B][F][NF] complex64 = interleaved (re, im) f32
 *               pairs, contiguous, 8-byte aligned (the alignment of a
 *               complex64 element; any contiguous view of a complex64
 *               tensor qualifies).                             (read-only)
 *   mel_filters device, [NM][NF] f32 row-major, 4-byte aligned; any dense
 *               matrix (only the span between the first and the last
 *               nonzero of each row is read).                  (read-only)
 *   out         device, [B][F][NM] f32, 4-byte aligned; must not overlap
 *               the inputs.
 *   B, F        clips and frames per clip (B, F >= 0; F may be ragged).
 *   NF, NM      bins per frame (1..8193) and mel bands (1..512).
 *   workspace   device, >= lm_log_mel_from_stft_workspace_size(B, F, NF, NM) bytes,
 *               4-byte aligned; its contents are overwritten.
 *
 * Errors: LM_ERR_INVALID_ARG (null pointer with B*F > 0, negative sizes),
 * LM_ERR_UNSUPPORTED (NF or NM out of range), LM_ERR_MISALIGNED (stft not
 * 8-byte aligned, out or workspace not 4-byte aligned), LM_ERR_WORKSPACE,
 * LM_ERR_CUDA.  B == 0 or F == 0 returns LM_OK and enqueues nothing.
 * Concurrent calls must use distinct workspaces.
 */
lm_status lm_log_mel_from_stft(const void *stft, const float *mel_filters, float *out, int64_t B,
                               int64_t F, int32_t NF, int32_t NM, void *workspace,
                               size_t workspace_bytes, lm_stream_t stream);

/* How lm_log_mel_from_stft will run a problem of this shape on the current
 * device (pure host-side planning; no work is enqueued).  Fields:
 *   resident       1 = single cooperative launch, one persistent CTA per SM,
 *                  that keeps each tile's log values on chip until its clip
 *                  maximum is known and writes the output once.
 *   cluster        > 0 = single launch of one thread-block cluster of this
 *                  many CTAs per clip (small batches, when the device runs
 *                  every clip's cluster at once): each CTA keeps its share
 *                  of the clip's log values in shared memory, the cluster
 *                  exchanges maxima through distributed shared memory, and
 *                  the output is written once.
 *                  resident = 0 and cluster = 0: two launches (log values,
 *                  then the in-place floor/rescale pass).
 *   kernels        kernel launches per call (1 or 2; plus one memset of the
 *                  workspace).
 *   grid           CTAs of the main kernel.
 *   frames_per_tile, stages, lag: tile height, shared-memory ring depth, and
 *                  how many tiles each thread holds back before writing.
 *   smem_bytes     dynamic shared memory per CTA.
 * LOGMEL_K1_VARIANT=resident|twopass|cluster forces a variant, and
 * =nocluster leaves the cluster variant out (A/B), and LOGMEL_FPB=1|2|4|6|8
 * forces the frames each consumer thread takes per tile (the workspace size
 * follows it); a forced variant or tile that cannot run returns
 * LM_ERR_UNSUPPORTED. */
typedef struct lm_stft_launch_info {
  int32_t resident;
  int32_t kernels;
  int32_t grid;
  int32_t frames_per_tile;
  int32_t stages;
  int32_t lag;
  int64_t smem_bytes;
  int32_t cluster;
  int32_t reserved;
} lm_stft_launch_info;

lm_status lm_log_mel_from_stft_describe(int64_t B, int64_t F, int32_t NF, int32_t NM,
                                        lm_stft_launch_info *info);

/* ---- Pre-packed filters (the "flashmel" page, "How it works": triangular
 * filters packed as start / width / weights) ----
 *
 * lm_log_mel_from_stft derives each band's support (first..last nonzero bin of
 * its row of the dense matrix) and first weights on every call; at kernel
 * start that costs a sweep of the whole matrix plus a second round of loads,
 * several microseconds that dominate small batches.  A caller that reuses
 * one filter matrix can pack it once and pass the pack:
 *
 *   lm_mel_filters_pack_size(NF, NM, &bytes)   bytes of device memory a pack
 *                                              needs (LM_ERR_INVALID_ARG /
 *                                              LM_ERR_UNSUPPORTED as for the
 *                                              shapes of lm_log_mel_from_stft).
 *   lm_mel_filters_pack(mel_filters, NF, NM, packed, bytes, stream)
 *       enqueues on `stream` the packing of the dense [NM][NF] f32 matrix
 *       (device, 4-byte aligned, read-only) into `packed` (device, caller
 *       owned, 16-byte aligned, >= the size above): a header with the shape,
 *       then {first bin, width} per band, then each band's first 8 weights
 *       from its first bin (zero past the width).  Errors:
 *       LM_ERR_INVALID_ARG (null), LM_ERR_MISALIGNED, LM_ERR_WORKSPACE (too
 *       small), LM_ERR_CUDA.
 *   lm_log_mel_from_stft_packed(stft, mel_filters, packed, out, ...)
 *       the same computation, arguments and results as lm_log_mel_from_stft,
 *       reading supports and first weights from `packed` (which must be made
 *       from this mel_filters, and be complete in stream order; bands wider
 *       than 8 bins still read the rest from mel_filters).  A pack whose
 *       header does not match NF, NM is not used: the call falls back to the
 *       dense matrix and sets bit 4 of the device error word
 *       (lm_workspace_error).  Errors: as lm_log_mel_from_stft, plus
 *       LM_ERR_INVALID_ARG for a null pack and LM_ERR_MISALIGNED for one not
 *       16-byte aligned.
 */
lm_status lm_mel_filters_pack_size(int32_t NF, int32_t NM, size_t *bytes);
lm_status lm_mel_filters_pack(const float *mel_filters, int32_t NF, int32_t NM, void *packed,
                              size_t packed_bytes, lm_stream_t stream);
lm_status lm_log_mel_from_stft_packed(const void *stft, const float *mel_filters, const void *packed,
                                      float *out, int64_t B, int64_t F, int32_t NF, int32_t NM,
                                      void *workspace, size_t workspace_bytes, lm_stream_t stream);

/* ---- Allocation-free variant (the source pages have no counterpart) ----
 *
 * Same computation, arguments and results as lm_log_mel_from_stft, without
 * the workspace argument.  It is meant for callers that cannot allocate
 * device memory themselves: code on a real-time audio thread, where a
 * cudaMalloc may block or synchronise the whole device, or a host
 * application that owns every byte of device memory and has no scratch to
 * hand out.
 *
 * Scratch comes from one fixed array of LM_NOALLOC_SCRATCH_BYTES compiled
 * into the library; every GPU that loads the library holds that array until
 * the process exits.  The call allocates and frees nothing.
 *  - Its first LM_NOALLOC_SCRATCH_BYTES - 256 bytes stand in for the
 *    workspace.  A problem needing more than that (about 16 bytes plus 4
 *    bytes per tile of frames; for NF = 201, NM = 128 a tile is 25 frames,
 *    so up to about 262,000 tiles, e.g. 256 clips of up to 25,500 frames)
 *    returns LM_ERR_WORKSPACE and enqueues nothing.
 *  - The first call on each device looks up the array's device address
 *    (cudaGetSymbolAddress) with that device current; make that first call
 *    before any stream capture.  The address is kept for the life of the
 *    process: after a cudaDeviceReset of that device it is stale, so do not
 *    call these entry points after one.
 *  - Every call uses the same array, which keeps the previous call's
 *    contents; each call clears the part it needs before its kernel runs.
 *    Calls whose work can overlap on the GPU (different streams, or host
 *    threads without ordering between them) race on the array: the caller
 *    must order them.
 *  - The kernels' device error bits go to a word in the array's last 256
 *    bytes, which no call clears: bits accumulate over calls until
 *    lm_log_mel_from_stft_noalloc_error reads and clears them.
 */
#define LM_NOALLOC_SCRATCH_BYTES (1u << 20)

lm_status lm_log_mel_from_stft_noalloc(const void *stft, const float *mel_filters, float *out,
                                       int64_t B, int64_t F, int32_t NF, int32_t NM,
                                       lm_stream_t stream);

/* Synchronises `stream`, then reads the accumulated device error word of
 * lm_log_mel_from_stft_noalloc calls on the current device (0 = no kernel
 * reported a problem) into *device_error, and clears it when `clear` is
 * nonzero (the clearing is ordered on `stream`).  Allocates nothing.
 * Returns LM_ERR_DEVICE_FAULT when the word was nonzero, LM_ERR_INVALID_ARG
 * for a null pointer, LM_ERR_CUDA when a CUDA call failed. */
lm_status lm_log_mel_from_stft_noalloc_error(uint32_t *device_error, int32_t clear, lm_stream_t stream);

/* Synchronises `stream`, then reads the device error word of a workspace
 * used by lm_log_mel_from_stft or lm_mel_spectrogram.  *device_error = 0
 * means no kernel reported a problem; otherwise it holds bit flags:
 *   1  an mbarrier wait inside a kernel ran out (2 s)
 *   2  waiting for another CTA's result ran out (a clip's maximum, or
 *      the launch token of the CTA that clears the workspace)
 *   4  a filter pack did not match the call (the dense matrix was used)
 *   8  (only in the bounds-checked debug build, compiled with
 *      -DLOGMEL_CHECKED) a computed global-memory index fell outside its
 *      buffer; the access was skipped
 * Returns LM_ERR_DEVICE_FAULT when it is nonzero. */
lm_status lm_workspace_error(const void *workspace, size_t workspace_bytes, uint32_t *device_error,
                             lm_stream_t stream);

/* ---- Fault injection for tests of the bounded waits (the source pages
 * have no counterpart) ----
 *
 * Runs lm_log_mel_from_stft on its one-CTA-per-SM kernel (same arguments,
 * results and errors; the cluster variant has no cross-CTA waits) with two
 * changes that make one of its cross-CTA waits run out on purpose, so that
 * a test can check that the kernel gives up cleanly instead of hanging:
 *   withheld_tile  the maximum of this tile of frames is never published
 *                  (tiles are numbered clip by clip; a clip has
 *                  ceil(F / frames_per_tile) of them, see
 *                  lm_log_mel_from_stft_describe); >= 0.
 *   clip_wait_ns   how long a CTA waits for a clip's maximum before giving
 *                  up (the regular calls wait 2 s); 1e5 .. 2e9.
 * When a wait gives up, the CTA sets bit 2 of the workspace's device error
 * word, its warps stop without further stores, and it exits once its
 * in-flight copies have landed.  The outputs of the clip whose tile was
 * withheld (and, where a CTA ran tiles of several clips, of the clips it
 * had not finished) are left incomplete.  Only single-kernel (resident)
 * launches wait across CTAs; for two-launch shapes the tile's slot stays
 * zero and the epilogue reduces the clip maximum over the other tiles.
 * Returns LM_ERR_INVALID_ARG for arguments out of range. */
lm_status lm_debug_log_mel_from_stft_withhold(const void *stft, const float *mel_filters, float *out,
                                              int64_t B, int64_t F, int32_t NF, int32_t NM, void *workspace,
                                              size_t workspace_bytes, int64_t withheld_tile,
                                              uint64_t clip_wait_ns, lm_stream_t stream);

/* ------------------------------------------------------------------------ */
/* 2. waveform -> mel spectrogram                                            */
/* ------------------------------------------------------------------------ */

/* Parameters of a mel spectrogram, named as torchaudio's MelSpectrogram
 * arguments listed on the flashmel page (window is always periodic Hann,
 * onesided always true). */
typedef struct lm_mel_params {
  int32_t sample_rate; /* Hz, > 0 */
  int32_t n_fft;       /* 400, or a power of two in [64, 16384] */
  int32_t win_length;  /* 0 = n_fft; otherwise 1..n_fft, window centred in the frame */
  int32_t hop_length;  /* > 0 */
  int32_t n_mels;      /* 1..256 */
  float f_min;         /* Hz, >= 0 */
  float f_max;         /* Hz, > f_min; <= 0 means sample_rate / 2 */
  int32_t pad;         /* zeros added on both sides before centre padding, >= 0 */
  int32_t center;      /* 1: pad n_fft/2 on both sides with pad_mode */
  int32_t pad_mode;    /* lm_pad_mode */
  float power;         /* 1 (magnitude) or 2 (power) */
  int32_t normalized;  /* 1: scale the window by 1/sqrt(sum w^2) */
  int32_t mel_scale;   /* lm_mel_scale */
  int32_t slaney_norm; /* 1: each triangle scaled to unit area */
  int32_t log_mel;     /* 1: log10(max(x,1e-10)), per-clip clamp at max-8, (x+4)/4 */
} lm_mel_params;

typedef struct lm_mel_plan lm_mel_plan;

/* Validates `params`, builds the window, filterbank and FFT tables on the
 * host in double and uploads them (rounded to f32) to the current device.
 * Errors: LM_ERR_INVALID_ARG, LM_ERR_UNSUPPORTED, LM_ERR_OUT_OF_MEMORY,
 * LM_ERR_CUDA; on any error *plan is NULL and nothing stays allocated.
 * The plan is immutable and may be shared by streams.
 * For tests of that error path, the environment variable
 * LOGMEL_FAULT=plan_alloc (or plan_alloc:k) makes the first (k-th) of the
 * plan's device allocations fail as if the device were out of memory. */
lm_status lm_mel_plan_create(const lm_mel_params *params, lm_mel_plan **plan);

/* Frees the plan's device tables (synchronises the device first). */
lm_status lm_mel_plan_destroy(lm_mel_plan *plan);

/* Number of output frames for a signal of T samples. */
lm_status lm_mel_n_frames(const lm_mel_plan *plan, int64_t T, int64_t *n_frames);

/* Bytes of device workspace lm_mel_spectrogram needs for B clips of T
 * samples (a header and, for log plans, one u32 per tile of frames and two
 * per clip). */
lm_status lm_mel_workspace_size(const lm_mel_plan *plan, int64_t B, int64_t T, size_t *bytes);

/*
 * Mel spectrogram of B waveforms (flashmel page, usage and "how it works").
 *
 *   wave      device, [B][T] f32 (in_dtype LM_F32) or int16 (LM_I16, scaled
 *             by 1/32768), contiguous, 4-byte aligned.          (read-only)
 *   out       device, [B][n_mels][n_frames] f32 (LM_F32) or f16 (LM_F16),
 *             4-byte aligned.  log_mel plans require LM_F32.
 *   workspace device, >= lm_mel_workspace_size(plan, B, T) bytes, 4-byte
 *             aligned; its contents on entry do not matter.  An 8-byte
 *             aligned workspace needs no memset before the kernel (the
 *             kernel clears its error word, tile counter and clip words
 *             itself, keyed by a per-launch token); a 4-byte aligned one,
 *             or any call made while the stream is being captured into a
 *             graph, gets a memset first.
 *
 * Log plans run as two launches: the transform, then a clamp-only kernel
 * launched as a programmatic dependent (its launch overlaps the first
 * kernel's tail).  With LOGMEL_K3_EPILOGUE=fused, where n_fft is 64, 128,
 * 256, 400, 512 or 1024, the clip floor and rescale are applied by the same
 * cooperative grid instead (one launch, the same bits; measured slower).
 * Non-log plans are one launch.
 *
 * Errors: LM_ERR_INVALID_ARG (null pointers, T too short for reflect
 * padding, n_frames < 1), LM_ERR_UNSUPPORTED (dtype combination),
 * LM_ERR_MISALIGNED, LM_ERR_WORKSPACE, LM_ERR_CUDA.
 */
lm_status lm_mel_spectrogram(const lm_mel_plan *plan, const void *wave, int32_t in_dtype, int64_t B,
                             int64_t T, void *out, int32_t out_dtype, void *workspace,
                             size_t workspace_bytes, lm_stream_t stream);

/* ------------------------------------------------------------------------ */
/* 3. host buffers in and out (the source pages have no counterpart)        */
/* ------------------------------------------------------------------------ */

/*
 * The same computations as lm_log_mel_from_stft(_packed) and
 * lm_mel_spectrogram, for inputs and results in host memory.  The library
 * cuts the batch into chunks of whole clips and pipelines them through
 * three staging slots in the workspace: the copy in of one chunk, the
 * kernels of the previous one and the copy out of the one before run at
 * the same time, on two internal streams of the library and `stream`.
 * Results equal those of the device entry points bit for bit (clips are
 * independent; the per-clip maximum never crosses a chunk).
 *
 *   stft_host / wave_host  host, laid out as the device entry point's input.
 *   out_host               host, laid out as the device entry point's output;
 *                          must not overlap the input.
 *                          Both should be page-locked (cudaHostAlloc or
 *                          cudaHostRegister) for the copies to overlap;
 *                          pageable memory gives the same results, with the
 *                          copies serialised and the call blocking the host.
 *   mel_filters, packed    device, as for lm_log_mel_from_stft_packed;
 *                          packed may be NULL (dense filters).
 *   chunk_clips            clips per chunk; 0 = the library's choice: whole
 *                          clips filling about 32 MB of input, and at most a
 *                          third of the batch (rounded up).
 *   workspace              device, 256-byte aligned, >= the matching
 *                          *_host_workspace_size (a 256-byte header whose
 *                          first u32 is the device error word of every
 *                          chunk, the operation's workspace for one chunk,
 *                          then three input and three output slots).
 *   stream                 the call is ordered on it: the copy streams
 *                          start after its earlier work, and it waits for
 *                          the last copy out.  out_host is complete once
 *                          `stream` reaches that point (e.g. after
 *                          cudaStreamSynchronize(stream)).
 *
 * The first call on a device, and each further call that overlaps in time
 * with the others, creates two streams and twelve events that the library
 * keeps for reuse until the process exits; no memory is allocated.
 *
 * Errors: as the device entry points, plus LM_ERR_INVALID_ARG when the host
 * buffers overlap, and LM_ERR_UNSUPPORTED when `stream` is capturing a
 * CUDA graph (the pipeline is not capturable).  Argument errors are found
 * before anything is enqueued; lm_workspace_error reads the error word.
 * Calls that overlap in time need distinct workspaces.
 */
lm_status lm_log_mel_from_stft_host_workspace_size(int64_t B, int64_t F, int32_t NF, int32_t NM,
                                                   int64_t chunk_clips, size_t *bytes);
lm_status lm_log_mel_from_stft_host(const void *stft_host, const float *mel_filters, const void *packed,
                                    float *out_host, int64_t B, int64_t F, int32_t NF, int32_t NM,
                                    int64_t chunk_clips, void *workspace, size_t workspace_bytes,
                                    lm_stream_t stream);

lm_status lm_mel_spectrogram_host_workspace_size(const lm_mel_plan *plan, int64_t B, int64_t T,
                                                 int32_t in_dtype, int32_t out_dtype, int64_t chunk_clips,
                                                 size_t *bytes);
lm_status lm_mel_spectrogram_host(const lm_mel_plan *plan, const void *wave_host, int32_t in_dtype,
                                  int64_t B, int64_t T, void *out_host, int32_t out_dtype,
                                  int64_t chunk_clips, void *workspace, size_t workspace_bytes,
                                  lm_stream_t stream);

/* ------------------------------------------------------------------------ */
/* 4. linear layers (the source pages have no counterpart)                  */
/* ------------------------------------------------------------------------ */

typedef enum lm_activation {
  LM_ACT_NONE = 0,
  LM_ACT_RELU = 1,      /* max(z, 0) */
  LM_ACT_GELU = 2,      /* z * (1 + erf(z / sqrt 2)) / 2 */
  LM_ACT_GELU_TANH = 3, /* z * (1 + tanh(sqrt(2/pi) * (z + 0.044715 z^3))) / 2 */
  LM_ACT_SILU = 4       /* z / (1 + exp(-z)) */
} lm_activation;

/*
 * y = residual + scale * act(x W^T + bias), for features and states of a
 * speech model that reads this library's log-mel frames.
 *
 *   x         device, [groups][rows][k], read through x_group_stride and
 *             x_row_stride (elements, >= 0; k contiguous).  Rows may overlap:
 *             a convolution over frames is a product with the windows of
 *             [frames][n_mels] read in place, k = taps * n_mels and
 *             x_row_stride = hop * n_mels.                      (read-only)
 *   weight    device, [n][k], weight_row_stride elements apart. (read-only)
 *   bias      device, [n] of bias_dtype, or NULL.               (read-only)
 *   residual  device, [groups*rows][n] of dtype, residual_row_stride
 *             elements apart, or NULL; may equal out (same row stride).
 *   out       device, [groups*rows][n] of out_dtype, out_row_stride
 *             elements apart (>= n); must not overlap the other inputs.
 *   dtype     LM_F16 or LM_BF16: type of x, weight and residual.
 *   bias_dtype  LM_F32 or dtype.
 *   out_dtype   dtype or LM_F32.
 *
 * Products are summed in 32 bits; bias, activation, scale and residual are
 * applied in 32 bits and rounded once to out_dtype.  k = 0 gives act(bias).
 * Pointers are aligned to their element.  An x or weight whose rows do not all
 * start on 16 bytes is copied into the workspace first.
 *
 *   workspace device, >= lm_linear_workspace_size(args), 16-byte aligned,
 *             filled with zeros before its first use; every call leaves the
 *             counters in it at zero, so calls of this function in stream
 *             order may share one.
 *             Its first u32 is the device error word (lm_workspace_error).
 *
 * Errors: LM_ERR_INVALID_ARG (null, negative sizes or strides, unknown
 * activation, overlapping rows of out), LM_ERR_UNSUPPORTED (dtypes; n, k or groups*rows >= 2^31),
 * LM_ERR_MISALIGNED, LM_ERR_WORKSPACE, LM_ERR_CUDA.  groups * rows * n == 0
 * returns LM_OK and enqueues nothing.
 */
typedef struct lm_linear_args {
  const void *x;
  const void *weight;
  const void *bias;
  const void *residual;
  void *out;
  int64_t groups, rows, k, n;
  int64_t x_group_stride, x_row_stride, weight_row_stride, residual_row_stride, out_row_stride;
  int32_t dtype, bias_dtype, out_dtype, activation;
  float scale;
  int32_t reserved;
} lm_linear_args;

lm_status lm_linear_workspace_size(const lm_linear_args *args, size_t *bytes);
lm_status lm_linear(const lm_linear_args *args, void *workspace, size_t workspace_bytes, lm_stream_t stream);

/* Synchronises `stream`, then reads the bits (those of lm_workspace_error)
 * that lm_linear, lm_linear4, lm_gated_linear, its backward pass and lm_kv_attend have reported on the current device, on any
 * stream and with any workspace, since the word was last cleared; clears it
 * where `clear` is nonzero.  Where it is not zero, some call's output is not
 * whole.  Returns LM_ERR_DEVICE_FAULT when a bit was set,
 * LM_ERR_INVALID_ARG for a null pointer, LM_ERR_CUDA when a CUDA call failed. */
lm_status lm_decode_error(uint32_t *device_error, int32_t clear, lm_stream_t stream);

/* Fault injection for tests of the bounded waits: lm_linear, except that the
 * first tile of operands that CTA `withheld_cta` (>= 0) fetches never counts as
 * complete, and that waits give up after wait_ns (1e5 .. 2e9; 2 s otherwise).
 * The CTA sets bit 1 of the workspace's error word and ends; its outputs are
 * not written (where CTAs share a tile's k, those of its tile are not right). */
lm_status lm_debug_linear_withhold(const lm_linear_args *args, void *workspace, size_t workspace_bytes,
                                   int64_t withheld_cta, uint64_t wait_ns, lm_stream_t stream);

/* ------------------------------------------------------------------------ */
/* 5. keys and values in 8 bits (the source pages have no counterpart)      */
/* ------------------------------------------------------------------------ */

/*
 * A cache of keys and values for `rows` sequences (a clip's encoder frames,
 * or a beam's tokens), held as signed 8-bit integers in blocks of `block`
 * tokens, with one f32 scale per layer, block and head:
 *     key = k8 * k_scale, value = v8 * v_scale.
 * Row r's token t is in place t % block of block table[r][t / block].
 *
 *   k8, v8            device, [layers][blocks][heads][block][head_dim] int8,
 *                     16-byte aligned
 *   k_scale, v_scale  device, [layers][blocks][heads] f32
 *   table             device, [rows][width] int32, block numbers.  An entry
 *                     outside [0, blocks) counts as tokens that are absent;
 *                     entries past a row's tokens are not used.
 *   spare             device, [rows] int32, one block per row that no table
 *                     entry names (lm_kv_reorder only; may be NULL otherwise)
 *   lens              device, [rows] int32, tokens held before this step
 *   head_dim          32, 64 or 128;  block 16, 32, 64 or 128
 *   rows              up to 65535 for lm_kv_read, lm_kv_attend and lm_kv_reorder
 * Rows hold at most width * block tokens: what a step adds past that is
 * dropped.  A negative length counts as 0.
 */
typedef struct lm_kv_cache {
  int8_t *k8;
  int8_t *v8;
  float *k_scale;
  float *v_scale;
  int32_t *table;
  int32_t *spare;
  int32_t *lens;
  int64_t blocks;
  int32_t layers, rows, width, heads, head_dim, block;
} lm_kv_cache;

/*
 * Appends tokens to one layer: row r's token i (i < counts[r], or < tokens
 * where counts is NULL) goes to place lens[r] + i.  lens itself is not
 * changed (every layer of a step appends at the same lengths).
 *   scale' = max(scale of what the block holds, max |new| * c), 1 where that
 *            is 0, with c the f32 nearest to 1 / 127 (so that scale' may be one
 *            unit in the last place off max |new| / 127);
 *   what the block holds: q' = rint(q * (scale / scale')) where it grew;
 *   new tokens:           q  = rint(x / scale').
 * Ties round to even.  A NaN or infinity among a block's new tokens makes its
 * scale infinite, so that the block's values read as NaN.
 *
 *   k, v     device, [rows][tokens][heads][head_dim] of dtype (LM_F16 or
 *            LM_BF16), read through k_strides and v_strides: elements
 *            between rows, tokens and heads; head_dim contiguous. (read-only)
 *   counts   device, [rows] int32 new tokens, clamped to [0, tokens]; or NULL
 *   k_values, v_values  both NULL, or device,
 *            [rows][span][heads][head_dim] of dtype, 16-byte aligned, with
 *            span = ((tokens - 1 + block - 1) / block + 1) * block:
 *            what the cache then holds from the first token of the block that
 *            lens[r] falls in; zeros past the row's last token.
 * A row's blocks must not be shared with another row from the block that
 * lens[r] falls in onwards.
 *
 * Errors: LM_ERR_INVALID_ARG, LM_ERR_UNSUPPORTED, LM_ERR_MISALIGNED,
 * LM_ERR_CUDA.  rows == 0 or tokens == 0 enqueues nothing.
 */
lm_status lm_kv_append(const lm_kv_cache *cache, int32_t layer, const void *k, const void *v,
                       const int64_t *k_strides, const int64_t *v_strides, int32_t tokens,
                       const int32_t *counts, int32_t dtype, void *k_values, void *v_values,
                       lm_stream_t stream);

/*
 * The values that tokens start .. start + count - 1 of every row stand for:
 * k_out, v_out device, [layers or 1][rows][count][heads][head_dim] of dtype,
 * 16-byte aligned; zeros from lens[r] on.  layer = -1 reads every layer.
 * Errors as lm_kv_append.
 */
lm_status lm_kv_read(const lm_kv_cache *cache, int32_t layer, int32_t start, int32_t count, int32_t dtype,
                     void *k_out, void *v_out, lm_stream_t stream);

/*
 * Attention over one layer of the cache, softmax(scale * q k^T) v per head.
 *   q        device, [rows][tokens][q_heads][head_dim] of dtype (LM_F16,
 *            LM_BF16), read through q_strides (rows, tokens, heads);
 *            q_heads a multiple of the cache's heads: query head h reads
 *            key head h / (q_heads / heads).                   (read-only)
 *   counts   device, [rows] int32 or NULL: new tokens of this step that the
 *            cache already holds past lens[r], at least 0, and at most
 *            `tokens` where causal is 1 (where it is 0, as many as the table
 *            holds: queries need not be those tokens'); NULL: new_tokens for
 *            every row.
 *   causal   1: query i stands at token lens[r] + i and sees tokens up to
 *            it; queries from counts[r] on see nothing.
 *            0: every query sees the lens[r] + counts[r] tokens.
 *   out      device, [rows][tokens][q_heads][head_dim] of dtype, contiguous,
 *            16-byte aligned.  A query that sees nothing gives zeros.
 *   workspace  device, >= lm_kv_attend_workspace_size(...), 16-byte aligned,
 *            zeroed before its first use, left usable by every call (as for
 *            lm_linear).
 * Scores, softmax statistics and the sums are held in 32 bits; a token's weight
 * is rounded to f16 (2^-11) on its way to the values.  Value scales count as at
 * least 2^-90.
 * Errors as lm_kv_append, and LM_ERR_WORKSPACE.
 */
lm_status lm_kv_attend_workspace_size(const lm_kv_cache *cache, int32_t tokens, int32_t q_heads, size_t *bytes);
lm_status lm_kv_attend(const lm_kv_cache *cache, int32_t layer, const void *q, const int64_t *q_strides,
                       int32_t tokens, int32_t q_heads, const int32_t *counts, int32_t new_tokens,
                       int32_t causal, float scale, int32_t dtype, void *out, void *workspace,
                       size_t workspace_bytes, lm_stream_t stream);

/* Fault injection for tests of the bounded waits: lm_kv_attend, except that
 * the first tile of tokens that CTA `withheld_cta` (>= 0, counted over the
 * grid) fetches never counts as complete, and that waits give up after
 * wait_ns (1e5 .. 2e9; 2 s otherwise).  A CTA whose wait runs out sets bit 1
 * of the workspace's error word, waits (bounded) for its copies and ends; the
 * outputs of its row, heads and queries are not written. */
lm_status lm_debug_kv_attend_withhold(const lm_kv_cache *cache, int32_t layer, const void *q, const int64_t *q_strides,
                                      int32_t tokens, int32_t q_heads, const int32_t *counts, int32_t new_tokens,
                                      int32_t causal, float scale, int32_t dtype, void *out, void *workspace,
                                      size_t workspace_bytes, int64_t withheld_cta, uint64_t wait_ns,
                                      lm_stream_t stream);

/* ------------------------------------------------------------------------ */
/* 6. beam search (the source pages have no counterpart)                    */
/* ------------------------------------------------------------------------ */

/*
 * One step of beam search: the `beams` best continuations of each clip.
 * Beam i of a clip offers its tokens at
 *     total = score[i] + ((x - max x) - log(sum exp(x - max x))),
 * x the beam's logits; a finished beam offers eos alone, at its score.
 * Best is the largest total; among equal totals the lower beam, then the
 * larger logit, then the lower token.  A beam whose logits hold a NaN or
 * +infinity, or nothing above -infinity, and a NaN total, count as -infinity
 * (places that nothing better fills are taken by such continuations).
 *
 *   logits    device, [clips][beams][vocab] of dtype (LM_F32, LM_F16,
 *             LM_BF16), rows row_stride elements apart.          (read-only)
 *   scores    device, [clips][beams] f32                         (read-only)
 *   finished  device, [clips][beams] u8 (0 or 1), or NULL: none  (read-only)
 *   history   device, [clips][beams][width] int32, or NULL       (read-only)
 *   length    place of the new token in the history, 0 <= length < width
 *   eos       the token that ends a beam; -1: none
 *   out_*     device, [clips][beams], best first: the totals f32, the tokens,
 *             the beams they continue (0 .. beams-1), and whether they have
 *             ended (u8): the continued beam had, or the token is eos.
 *   out_history  [clips][beams][width]: the continued beam's history with
 *             the token at `length` (NULL where history is); must not
 *             overlap history.
 *   beams     1..32;  vocab 1..2^24
 *   workspace device, >= lm_beam_step_workspace_size(...), 16-byte aligned,
 *             zeroed before its first use, left usable by every call.
 * Errors as above.  clips == 0 enqueues nothing.
 */
typedef struct lm_beam_args {
  const void *logits;
  const float *scores;
  const uint8_t *finished;
  const int32_t *history;
  float *out_scores;
  int32_t *out_tokens;
  int32_t *out_parents;
  uint8_t *out_finished;
  int32_t *out_history;
  int64_t clips, vocab, row_stride, width, length, eos;
  int32_t beams, dtype;
} lm_beam_args;

lm_status lm_beam_step_workspace_size(const lm_beam_args *args, size_t *bytes);
lm_status lm_beam_step(const lm_beam_args *args, void *workspace, size_t workspace_bytes, lm_stream_t stream);

/*
 * Lets the cache follow a beam step: rows are clips * beams, and row (c, i)
 * takes the tokens of row (c, parents[c][i]) (device, int32, each in
 * [0, beams); others leave their row as it is).  Rows of a clip have the
 * same length.  Whole blocks are shared by copying table entries; the block
 * that the next token falls in, where it holds tokens, is copied for every
 * layer into the row's spare block, which changes places with it.  A row
 * that continues itself is left alone.  An absent open block (table entry
 * outside [0, blocks)) stays absent in the rows that continue its row; a row
 * whose own is absent gives that entry to its spare when it continues another.
 *   workspace device, >= 16 + 4 * clips bytes, 16-byte aligned, zeroed before
 *             its first use, left usable by every call.
 * Errors as above, and LM_ERR_INVALID_ARG where spare is NULL or rows is not
 * a multiple of beams.
 */
lm_status lm_kv_reorder(const lm_kv_cache *cache, const int32_t *parents, int32_t beams, void *workspace,
                        size_t workspace_bytes, lm_stream_t stream);

/* ------------------------------------------------------------------------ */
/* 7. layer norm (the source pages have no counterpart)                     */
/* ------------------------------------------------------------------------ */

/*
 * y = (x - mean) / sqrt(var + eps) * weight + bias over the last dimension of
 * x [rows][width], with mean and var (the mean square of x - mean) of each row.
 *
 *   x        device, rows x_row_stride elements apart (>= 0: rows may overlap),
 *            of dtype LM_F32, LM_F16 or LM_BF16.                (read-only)
 *   weight, bias  device, [width], of weight_dtype and bias_dtype: LM_F32 or
 *            dtype; NULL: 1 and 0.                               (read-only)
 *   out      device, [rows][width] of dtype, rows out_row_stride elements
 *            apart; may be x itself (same stride), and meets no other input.
 *   stats    device, [3][rows] f32, or NULL: for lm_layer_norm_backward, the
 *            mean, what its rounding to f32 left off, and 1 / sqrt(var + eps).
 *   eps      >= 0
 * Sums are held in 32 bits, the deviations' taken about the rounded mean and put
 * right by theirs; y is rounded once.  A NaN or infinity in a row makes the row NaN.
 * Where the sum of a row's squared deviations passes 3.4e38 its y is bias, or NaN.
 *
 * Errors: LM_ERR_INVALID_ARG, LM_ERR_UNSUPPORTED (dtypes, sizes of 2^31 and
 * more), LM_ERR_MISALIGNED (pointers are aligned to their element), LM_ERR_CUDA.
 * rows * width == 0 enqueues nothing.
 */
typedef struct lm_norm_args {
  const void *x;
  const void *weight;
  const void *bias;
  void *out;
  float *stats;
  int64_t rows, width, x_row_stride, out_row_stride;
  int32_t dtype, weight_dtype, bias_dtype;
  float eps;
} lm_norm_args;

lm_status lm_layer_norm(const lm_norm_args *args, lm_stream_t stream);

/*
 * The gradients of lm_layer_norm.  With n = (x - mean) / sqrt(var + eps) and
 * h = grad * weight, row by row:
 *   dx = (h - avg(h) - n * avg(h * n)) / sqrt(var + eps)
 *   dweight = sum over rows of grad * n,   dbias = sum over rows of grad
 *
 *   x, weight, stats  as for (and from) lm_layer_norm
 *   grad     device, [rows][width] of dtype, rows grad_row_stride apart
 *   dx       device, [rows][width] of dtype, contiguous, or NULL: not wanted
 *   dweight  device, [width] of weight_dtype, or NULL
 *   dbias    device, [width] of bias_dtype, or NULL
 *   workspace  device, >= lm_layer_norm_backward_workspace_size(...), 16-byte
 *            aligned; its contents on entry do not matter.
 * Sums over rows are taken in 32 bits, in an order that depends on the sizes,
 * the rows' alignment and the device alone, and rounded once.  Outputs meet no input and not one another.
 * Errors as lm_layer_norm, and LM_ERR_WORKSPACE.  rows == 0 sets dweight and
 * dbias to zero.
 */
typedef struct lm_norm_backward_args {
  const void *x;
  const void *weight;
  const float *stats;
  const void *grad;
  void *dx;
  void *dweight;
  void *dbias;
  int64_t rows, width, x_row_stride, grad_row_stride;
  int32_t dtype, weight_dtype, bias_dtype, reserved;
} lm_norm_backward_args;

lm_status lm_layer_norm_backward_workspace_size(const lm_norm_backward_args *args, size_t *bytes);
lm_status lm_layer_norm_backward(const lm_norm_backward_args *args, void *workspace, size_t workspace_bytes,
                                 lm_stream_t stream);

/* ------------------------------------------------------------------------ */
/* 8. gated linear layers (the source pages have no counterpart)            */
/* ------------------------------------------------------------------------ */

#define LM_ACT_SIGMOID 5 /* 1 / (1 + exp(-z)); lm_gated_linear only */

/*
 * y = act(x Wg^T + bg) * (x Wu^T + bu): the first half of a gated feed-forward
 * block, both products, the activation and the product in one kernel.
 *
 *   x        device, [rows][k] of dtype (LM_F16, LM_BF16), rows x_row_stride
 *            elements apart (>= 0: rows may overlap), k contiguous. (read-only)
 *   w_gate, w_up  device, [n][k] of dtype, rows gate_row_stride and
 *            up_row_stride elements apart.                      (read-only)
 *   b_gate, b_up  device, [n] of bias_dtype (LM_F32 or dtype), or NULL each.
 *   out      device, [rows][n] of dtype, rows out_row_stride elements apart;
 *            meets no input.
 *   activation  one of lm_activation, or LM_ACT_SIGMOID
 * Products are summed in 32 bits, the rest is computed in 32 bits and rounded
 * once.  Operands whose rows do not all start on 16 bytes are copied into the
 * workspace first.
 *   workspace  device, >= lm_gated_linear_workspace_size(args), 16-byte aligned;
 *            its contents on entry do not matter but for the first u32, the
 *            device error word (lm_workspace_error), to which bits are added.
 *
 * Errors: LM_ERR_INVALID_ARG, LM_ERR_UNSUPPORTED (dtypes, sizes),
 * LM_ERR_MISALIGNED, LM_ERR_WORKSPACE, LM_ERR_CUDA.  rows * n == 0 enqueues
 * nothing.
 */
typedef struct lm_gated_args {
  const void *x;
  const void *w_gate;
  const void *w_up;
  const void *b_gate;
  const void *b_up;
  void *out;
  int64_t rows, k, n, x_row_stride, gate_row_stride, up_row_stride, out_row_stride;
  int32_t dtype, bias_dtype, activation, reserved;
} lm_gated_args;

lm_status lm_gated_linear_workspace_size(const lm_gated_args *args, size_t *bytes);
lm_status lm_gated_linear(const lm_gated_args *args, void *workspace, size_t workspace_bytes, lm_stream_t stream);

/*
 * The gradients of lm_gated_linear.  With a = x Wg^T + bg and b = x Wu^T + bu,
 * computed anew (nothing is kept from the forward pass but its inputs):
 *   da = grad * b * act'(a),   db = grad * act(a)
 *   dx = da Wg + db Wu,  dWg = da^T x,  dWu = db^T x,
 *   dbg, dbu = sums of da, db over rows
 * da and db are computed and, for the biases, summed in 32 bits, and rounded to
 * dtype as operands of the products (in f16 one past 65504 is infinite).  relu's
 * derivative at 0 is 0.  Each gradient's bits are the same whichever others are
 * wanted (but for db_gate and db_up where b_gate and b_up are both NULL).
 *
 *   forward  the inputs and sizes of lm_gated_linear (out and out_row_stride
 *            are not used)
 *   grad     device, [rows][n] of dtype, rows grad_row_stride elements apart
 *   dx [rows][k], dw_gate, dw_up [n][k] of dtype, db_gate, db_up [n] of
 *            bias_dtype: device, contiguous, each NULL where not wanted; they
 *            meet no input and not one another.
 *   workspace  as for lm_gated_linear, >= lm_gated_linear_backward_workspace_size(...)
 * Errors as lm_gated_linear.
 */
typedef struct lm_gated_backward_args {
  lm_gated_args forward;
  const void *grad;
  void *dx;
  void *dw_gate;
  void *dw_up;
  void *db_gate;
  void *db_up;
  int64_t grad_row_stride;
} lm_gated_backward_args;

lm_status lm_gated_linear_backward_workspace_size(const lm_gated_backward_args *args, size_t *bytes);
lm_status lm_gated_linear_backward(const lm_gated_backward_args *args, void *workspace, size_t workspace_bytes,
                                   lm_stream_t stream);

/* Fault injection for tests of the bounded waits, as lm_debug_linear_withhold:
 * in each kernel of the call the first tile of operands that CTA
 * `withheld_cta` (>= 0) fetches never counts as complete. */
lm_status lm_debug_gated_linear_withhold(const lm_gated_args *args, void *workspace, size_t workspace_bytes,
                                         int64_t withheld_cta, uint64_t wait_ns, lm_stream_t stream);
lm_status lm_debug_gated_linear_backward_withhold(const lm_gated_backward_args *args, void *workspace,
                                                  size_t workspace_bytes, int64_t withheld_cta, uint64_t wait_ns,
                                                  lm_stream_t stream);

/* ------------------------------------------------------------------------ */
/* 9. weights in 4 bits (the source pages have no counterpart)              */
/* ------------------------------------------------------------------------ */

/*
 * A weight [n][k] as whole numbers of -8 .. 7 and one f32 scale for each row
 * and `group` consecutive k:  w[i][j] = q[i][j] * s[i][j / group].
 *   packed   device, 16-byte aligned, blocks of 128 rows by 64 k: ceil(n / 128) *
 *            ceil(k / 64) blocks of 4096 bytes, along k first.  A block is eight
 *            tiles of 16 rows, 512 bytes each.
 *            Bytes 16 l .. 16 l + 15 of a tile are four little-endian u32 of
 *            eight k each: row l / 4 at k = 8 (l % 4) .. + 7 and 32 + 8 (l % 4) .. + 7,
 *            then row l / 4 + 8 at the same.  From a u32's lowest nibble the eight
 *            are in order 0 2 4 6 1 3 5 7; a nibble is q + 8.  Places past n or k
 *            hold q = 0.
 *   scale    device, [ceil(n / 128)][ceil(k / group)][128] f32, 16-byte aligned
 *   group    32, 64 or 128
 */
typedef struct lm_weight4 {
  const void *packed;
  const float *scale;
  int64_t n, k;
  int32_t group, reserved;
} lm_weight4;

/* Bytes of `packed` and `scale` for a weight of n, k and group. */
lm_status lm_weight4_size(const lm_weight4 *w, size_t *packed_bytes, size_t *scale_bytes);

/* Lays out q (device, int8 [n][k], contiguous, values clamped to -8 .. 7) and
 * scales (device, f32 [n][ceil(k / group)], contiguous) in w->packed and w->scale. */
lm_status lm_weight4_pack(const lm_weight4 *w, const int8_t *q, const float *scales, lm_stream_t stream);

/* Rounds weight (device, [n][k] of dtype LM_F32, LM_F16 or LM_BF16, rows
 * row_stride elements apart): s = max |w| of the group / 7 (1 where that is 0),
 * q = rint(w / s), ties to even.  A group with a NaN or infinity gets a scale of NaN or
 * infinity. */
lm_status lm_weight4_quantize(const lm_weight4 *w, const void *weight, int64_t row_stride, int32_t dtype,
                              lm_stream_t stream);

/* The values q * s, rounded to dtype (LM_F32, LM_F16, LM_BF16): out [n][k],
 * rows row_stride elements apart. */
lm_status lm_weight4_values(const lm_weight4 *w, void *out, int64_t row_stride, int32_t dtype, lm_stream_t stream);

/*
 * lm_linear with such a weight: args as there, but for weight and
 * weight_row_stride, which are not used; args->n and args->k are the weight's.
 * For few rows (up to 16; up to 64 where ceil(rows / 16) * n is at most 16384, 12000 for
 * k above 1024) a group's products q * x are summed in 32 bits and the sums multiplied by its scale.  For more the
 * values are rounded to dtype on their way into the products (to within 17/16
 * of half a step: the scale is taken in two parts of dtype); for many
 * (lm_linear4_expands) they are expanded into the workspace for lm_linear.
 *   workspace  as for lm_linear, >= lm_linear4_workspace_size(...)
 * Errors as lm_linear.
 */
lm_status lm_linear4_workspace_size(const lm_linear_args *args, const lm_weight4 *w, size_t *bytes);
lm_status lm_linear4(const lm_linear_args *args, const lm_weight4 *w, void *workspace, size_t workspace_bytes,
                     lm_stream_t stream);
/* Fault injection for tests of the bounded waits, as lm_debug_linear_withhold. */
lm_status lm_debug_linear4_withhold(const lm_linear_args *args, const lm_weight4 *w, void *workspace,
                                    size_t workspace_bytes, int64_t withheld_cta, uint64_t wait_ns, lm_stream_t stream);
/* 1 where a call with these sizes expands the weight, 0 where it reads the 4 bits in its products. */
int lm_linear4_expands(int64_t rows, int64_t n, int64_t k);

#ifdef __cplusplus
}
#endif

#endif /* LOGMEL_H_ */
