/*
 * rlca.h -- C ABI of the MI355X (gfx950) credit-assignment scan library.
 *
 * Seven reinforcement-learning credit-assignment estimators computed as one
 * first-order affine recurrence over [num_envs, T] rollouts:
 *   backward  A_t = alpha_t + beta_t * A_{t+1}   (GAE, TD(lambda), discounted
 *             returns, V-Trace, Retrace(lambda))
 *   forward   A_t = alpha_t + beta_t * A_{t-1}   (eligibility traces, episodic
 *             prefix sums)
 * ("rl-triton: High-Performance Triton GPU Kernels for Reinforcement Learning
 * Credit Assignment", paperlayer.ai summary, §1 Introduction and §3.1 Shared
 * scan formulation).  Each estimator call is one kernel launch that reads
 * its inputs from HBM once and writes each output once -- except for few
 * long rows (fewer than 128 rows of 16384 steps or more; for the forward
 * scans fewer than 160 rows of 32768 steps or more and fewer than 208 from
 * 65536 steps on), where each row is split into chunks that run in
 * parallel: three launches, inputs read twice, and the first
 * output array holds the chunk hand-off values until the last launch
 * overwrites them.  The fused consumers of GAE at the end of this header
 * are one launch each too.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Memory:  every array argument is a DEVICE pointer (hipMalloc memory or a
 *          torch tensor's data_ptr()) owned by the caller.  The library
 *          allocates nothing, keeps no mutable global state and never
 *          synchronizes: work is enqueued on `stream` and buffers must stay
 *          alive until the stream has passed the call.  With no state
 *          between calls, any entry point may be called from several host
 *          threads at once, on one stream or on several; only calls whose
 *          outputs overlap each other or another call's inputs, with nothing
 *          ordering them, race.
 * Layout:  per-step arrays are dense row-major [num_envs, T]; element (n, t)
 *          is at n*T + t.  `bootstrap` is [num_envs].  Real-valued and int32
 *          data must be aligned to its element size.  Flags are one byte per
 *          step, any nonzero byte meaning "set" (torch.bool and uint8 both
 *          work).  Speed, not results, depends on where arrays start: call
 *          an array's phase its start address's element index mod 4 from a
 *          four-element boundary (16 bytes for fp32, 8 for bf16 / fp16, 4
 *          for flags).  Every per-step array at phase 0 with T % 4 == 0 is
 *          the fastest case; per-step inputs all at one phase take the
 *          vectorised path too (outputs at another phase are then written
 *          element by element); inputs at different phases are read element
 *          by element.  On the vectorised path, except in the fastest case,
 *          the library reads whole aligned four-element blocks: it may read
 *          (never write) up to three elements before the start or past the
 *          end of a per-step input, inside the aligned block that holds its
 *          first or last element.  Such reads cannot fault and their values
 *          are not used.
 * Episode boundaries (summary §3.2 Episode-boundary semantics):
 *          terminated[t]  the episode ends after step t in a terminal state:
 *                         successor value 0, no credit flows back past t.
 *          truncated[t]   the episode is cut after step t (time limit): the
 *                         successor value is trunc_values[t] (the value of the
 *                         state the episode was cut in), no credit flows back
 *                         past t.  Terminated wins when both are set.
 *                         truncated == NULL means no truncation and selects a
 *                         specialised fast path; trunc_values is then ignored.
 *          t = T-1        the rollout window ends: when the last step is not
 *                         done, its successor value is bootstrap[n]
 *                         (bootstrap == NULL means 0).  A done last step
 *                         ignores the bootstrap.
 * Errors:  the return value is the only error channel.  Arguments are checked
 *          before anything is enqueued and a failed call has no side effects.
 *            RLCA_ERR_NULL_POINTER   a required pointer is NULL
 *            RLCA_ERR_INVALID_SIZE   num_envs < 0, T < 0, T > RLCA_MAX_T,
 *                                    num_envs > RLCA_MAX_ENVS, the byte
 *                                    size of an array overflows, or the
 *                                    launch would need more than 2^31 - 1
 *                                    workgroups (only num_envs near
 *                                    RLCA_MAX_ENVS with rows longer than one
 *                                    tile: terabytes of input)
 *            RLCA_ERR_INVALID_VALUE  gamma or lambda outside [0, 1] or not
 *                                    finite, rho_bar <= 0 or not finite,
 *                                    c_bar outside (0, 1], an unknown enum
 *                                    value
 *            RLCA_ERR_ALIASING       an output overlaps an input or another
 *                                    output (in-place is not supported)
 *            RLCA_ERR_MISALIGNED     an array is not aligned to its element size
 *            RLCA_ERR_HIP            a kernel launch failed (its hipError_t)
 *          num_envs * T == 0 is a valid no-op.  Faults inside the kernel
 *          surface at the caller's next synchronisation, as usual in HIP.
 *          Non-finite inputs are not trapped; they propagate inside their
 *          episode segment only.  A chain cut (a terminated or truncated
 *          step, a row end, a forward reset, a coefficient of exactly 0,
 *          e.g. lambda = 0 or gamma = 0) stops them: a NaN or infinity in
 *          one row never reaches another row, and never crosses an episode
 *          boundary within its row.  Inside a segment they also stop where
 *          the product of the coefficients between two steps rounds to 0
 *          (after about 1,700 steps at gamma * lambda = 0.94 in fp32 scans,
 *          far later in fp64 ones).  A NaN log-probability gives a NaN
 *          importance weight (not a clamped one).
 * Numerics: fp32 arithmetic (the summary's §4 requires float32 scans),
 *          with the fp64 scans stated below where fp32 would miss the
 *          summary's tolerance; the scan reassociates the recurrence
 *          (associativity, summary §5), so results match a sequential fp64
 *          evaluation to rounding, not bit for bit.  The int32 prefix sum is exact
 *          (two's-complement wrap).  Arrays may instead be stored as bf16 or
 *          fp16 (rlca_dtype; the summary's §9 defers bfloat16 I/O): they are
 *          widened exactly to fp32 on load and every output is rounded once,
 *          to nearest even, on store.  Every estimator's coefficient is a
 *          contraction, 0 <= beta_t <= 1 (gamma, lambda in [0, 1] and trace
 *          clips c_bar <= 1).  Where a chain that barely decays (beta near 1)
 *          carries a value across the 256-step waves of the scan, fp32
 *          rounding of the beta products and of the carried sums would
 *          build up along the row; such calls (and every generic affine
 *          scan over rows longer than 256 steps) scan in fp64 and round
 *          each output once, so chains that never break (a prefix sum
 *          without resets, gamma = 1 returns) keep their accuracy over the
 *          row, 131072 steps and more.  Affine coefficients beyond +-1 let
 *          products of beta grow, and rounding errors grow with them in
 *          any evaluation order; 16-bit storage may then overflow.
 */
#ifndef RLCA_H
#define RLCA_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define RLCA_MAX_T ((int64_t)1 << 30)
#define RLCA_MAX_ENVS ((int64_t)1 << 31)

/* Clamp applied to log(pi/mu) before exp() in V-Trace and Retrace. */
#define RLCA_LOG_RATIO_CLIP 5.0f

typedef enum {
    RLCA_OK = 0,
    RLCA_ERR_NULL_POINTER = 1,
    RLCA_ERR_INVALID_SIZE = 2,
    RLCA_ERR_INVALID_VALUE = 3,
    RLCA_ERR_ALIASING = 4,
    RLCA_ERR_MISALIGNED = 5,
    RLCA_ERR_HIP = 6
} rlca_status;

/* Forward-scan reset conventions.  The summary's §3.3 leaves the boundary
 * convention of the segmented forward scans configurable; its §5 cuts the
 * forward carry at the step after a done step. */
typedef enum {
    RLCA_RESET_ON_START = 0,  /* flags[t] != 0: step t starts a new episode      */
    RLCA_RESET_AFTER_DONE = 1 /* flags[t-1] != 0: step t-1 ended the episode      */
} rlca_reset_convention;

/* Element type of the data arrays.  RLCA_F32, RLCA_BF16 and RLCA_F16 are
 * storage types of the real-valued arrays (arithmetic is fp32 for all
 * three); RLCA_I32 is the exact integer prefix sum. */
typedef enum { RLCA_F32 = 0, RLCA_I32 = 1, RLCA_BF16 = 2, RLCA_F16 = 3 } rlca_dtype;

typedef enum { RLCA_BACKWARD = 0, RLCA_FORWARD = 1 } rlca_direction;

/* Generalized advantage estimation (Schulman et al. 2016; summary §2.1).
 *   delta_t = r_t + gamma * V(s_{t+1}) - V(s_t),   V(s_{t+1}) per the boundary rules
 *   adv_t   = delta_t + gamma * lambda * adv_{t+1}  (chain cut at done steps and t = T-1)
 *   ret_t   = adv_t + V(s_t)
 * rewards, values [N,T] f32; terminated [N,T] u8 (required); truncated [N,T] u8
 * (nullable); trunc_values [N,T] f32 (required iff truncated); bootstrap [N]
 * f32 (nullable).  Writes advantages [N,T] and, when non-NULL, returns [N,T]. */
rlca_status rlca_gae(const float *rewards, const float *values, const uint8_t *terminated,
                     const uint8_t *truncated, const float *trunc_values,
                     const float *bootstrap, float gamma, float lambda, int64_t num_envs,
                     int64_t T, float *advantages, float *returns, hipStream_t stream);

/* TD(lambda) returns (summary §1, §3.2):
 *   G_t = r_t + gamma * ((1 - lambda) * V(s_{t+1}) + lambda * G_{t+1}),
 *   and G_t = r_t + gamma * successor value at a done step or at t = T-1.
 * Arguments as rlca_gae; writes returns [N,T]. */
rlca_status rlca_td_lambda(const float *rewards, const float *values,
                           const uint8_t *terminated, const uint8_t *truncated,
                           const float *trunc_values, const float *bootstrap, float gamma,
                           float lambda, int64_t num_envs, int64_t T, float *returns,
                           hipStream_t stream);

/* Discounted returns (summary §1, §3.2): G_t = r_t + gamma * G_{t+1}, and
 * G_t = r_t + gamma * successor value at a done step or at t = T-1
 * (bootstrap == NULL gives Monte-Carlo returns).  Writes returns [N,T]. */
rlca_status rlca_discounted_returns(const float *rewards, const uint8_t *terminated,
                                    const uint8_t *truncated, const float *trunc_values,
                                    const float *bootstrap, float gamma, int64_t num_envs,
                                    int64_t T, float *returns, hipStream_t stream);

/* V-Trace (Espeholt et al. 2018; summary §8 Off-policy correction).
 *   ratio_t = exp(clamp(target_logp_t - behaviour_logp_t, -5, 5))
 *   rho_t = min(rho_bar, ratio_t),  c_t = lambda * min(c_bar, ratio_t)
 *   vs_t - V_t = rho_t (r_t + gamma V(s_{t+1}) - V_t) + gamma c_t (vs_{t+1} - V_{t+1})
 *   pg_t = rho_t (r_t + gamma vs_{t+1} - V_t)
 * where at a done step or t = T-1 the successor value replaces V(s_{t+1}) and
 * vs_{t+1}.  lambda = 1 is the IMPALA form.  rho_bar > 0; 0 < c_bar <= 1 (a
 * trace clip above 1 would make the recurrence expansive). 
 * Writes vs [N,T] and, when non-NULL, pg_advantages [N,T]. */
rlca_status rlca_vtrace(const float *rewards, const float *values, const float *behaviour_logp,
                        const float *target_logp, const uint8_t *terminated,
                        const uint8_t *truncated, const float *trunc_values,
                        const float *bootstrap, float gamma, float lambda, float rho_bar,
                        float c_bar, int64_t num_envs, int64_t T, float *vs,
                        float *pg_advantages, hipStream_t stream);

/* Retrace(lambda) (Munos et al. 2016; summary §3.3: the decay uses the
 * next step's importance weight).
 *   c_t = lambda * min(c_bar, exp(clamp(target_logp_t - behaviour_logp_t, -5, 5)))
 *   Qret_t = r_t + gamma E_pi Q(s_{t+1}, .) + gamma c_{t+1} (Qret_{t+1} - Q_{t+1})
 * q_values[t] = Q(s_t, a_t); expected_q[t] = E_pi Q(s_t, .).  At a done step
 * or t = T-1 the successor value (0 / trunc_values[t] = E_pi Q of the cut
 * state / bootstrap[n] = E_pi Q(s_T, .)) replaces E_pi Q(s_{t+1}, .) and the
 * correction term is dropped.  0 < c_bar <= 1 (Munos et al. truncate the
 * trace at 1).  Writes q_ret [N,T]. */
rlca_status rlca_retrace(const float *rewards, const float *q_values, const float *expected_q,
                         const float *behaviour_logp, const float *target_logp,
                         const uint8_t *terminated, const uint8_t *truncated,
                         const float *trunc_values, const float *bootstrap, float gamma,
                         float lambda, float c_bar, int64_t num_envs, int64_t T,
                         float *q_ret, hipStream_t stream);

/* Accumulating eligibility traces, forward in time (summary §1, §3.2):
 *   e_t = x_t + gamma * lambda * e_{t-1},  e_{-1} = 0, and e_{t-1} := 0 where
 *   a new episode starts under `convention`.
 * increments [N,T] f32, flags [N,T] u8 (required).  Writes traces [N,T]. */
rlca_status rlca_eligibility_traces(const float *increments, const uint8_t *flags,
                                    rlca_reset_convention convention, float gamma,
                                    float lambda, int64_t num_envs, int64_t T, float *traces,
                                    hipStream_t stream);

/* Inclusive episodic (segmented) prefix sum, forward in time (summary §3.3):
 *   S_t = x_t + S_{t-1},  S_{-1} = 0, restarted where a new episode starts.
 * x and out are [N,T] of `dtype` (f32, bf16 or f16; or i32 with
 * two's-complement wrap-around, exact); flags [N,T] u8 (required). */
rlca_status rlca_episodic_prefix_sum(const void *x, rlca_dtype dtype, const uint8_t *flags,
                                     rlca_reset_convention convention, int64_t num_envs,
                                     int64_t T, void *out, hipStream_t stream);

/* Generic first-order affine scan over caller-built coefficients (the
 * summary's §4 Scan procedure: the generic kernel that takes precomputed
 * alpha and beta instead of building them from a rollout).
 *   RLCA_BACKWARD: A_t = alpha_t + beta_t * A_{t+1},  A_T = carry[n]
 *   RLCA_FORWARD:  A_t = alpha_t + beta_t * A_{t-1},  A_{-1} = carry[n]
 * alpha, beta, out [N,T] f32; carry [N] f32, nullable (=> 0).  Episode
 * boundaries are the caller's business (beta_t = 0 cuts the chain).  Writes
 * out [N,T]. */
rlca_status rlca_affine_scan(const float *alpha, const float *beta, const float *carry,
                             rlca_direction direction, int64_t num_envs, int64_t T, float *out,
                             hipStream_t stream);

/* ---------------------------------------------------------------- batches
 * Several of the calls above enqueued together.  Each element is validated
 * exactly as its own entry point would validate it (the same status codes,
 * nothing enqueued on any failure), plus: no call may write memory that
 * another call of the batch reads or writes (RLCA_ERR_ALIASING), because the
 * calls run concurrently.  Calls on the vectorised path that need a single
 * launch share grouped launches (one launch for up to 14 calls of one shape
 * class and storage type), which removes the per-launch overhead that
 * dominates small rollouts; the others are enqueued one by one.  Results
 * are bit for bit those of the separate calls (a grouped launch keeps each
 * call's tile geometry).
 * (Launch-overhead reduction for small shapes: the summary's §9
 * Limitations, where launch and wrapper overhead dominate at 16 steps.) */
#define RLCA_MAX_BATCH 64

typedef enum {
    RLCA_OP_GAE = 0,
    RLCA_OP_TD_LAMBDA = 1,
    RLCA_OP_DISCOUNTED_RETURNS = 2,
    RLCA_OP_VTRACE = 3,
    RLCA_OP_RETRACE = 4,
    RLCA_OP_ELIGIBILITY_TRACES = 5,
    RLCA_OP_EPISODIC_PREFIX_SUM = 6,
    RLCA_OP_AFFINE_SCAN = 7
} rlca_op;

/* One call of a batch.  Fields carry the arguments of the op's entry point;
 * fields an op does not take are ignored.
 *   rewards     rewards (GAE, TD, discounted, V-Trace, Retrace); increments
 *               (eligibility traces); x (prefix sum); alpha (affine scan)
 *   values      values (GAE, TD, V-Trace); q_values (Retrace); beta (affine)
 *   terminated  terminated (backward estimators); flags (forward scans)
 *   bootstrap   bootstrap (backward estimators); carry (affine scan)
 *   out0        advantages / returns / vs / q_ret / traces / out
 *   out1        GAE returns or V-Trace pg_advantages; nullable
 *   dtype       element type of every real-valued array of the call, inputs
 *               and outputs alike: RLCA_F32 (0), RLCA_BF16 or RLCA_F16; the
 *               prefix sum also takes RLCA_I32.  This is how the bf16 / fp16
 *               forms of every op are reached (the single-call entry points
 *               above are fp32, except the prefix sum, which takes dtype).
 *   convention, direction: as the forward scans / affine scan take them */
typedef struct {
    rlca_op op;
    int64_t num_envs;
    int64_t T;
    const void *rewards;
    const void *values;
    const void *expected_q;
    const void *behaviour_logp;
    const void *target_logp;
    const uint8_t *terminated;
    const uint8_t *truncated;
    const void *trunc_values;
    const void *bootstrap;
    float gamma;
    float lambda;
    float rho_bar;
    float c_bar;
    int convention;
    int dtype;
    int direction;
    void *out0;
    void *out1;
} rlca_call;

/* Enqueue `count` (0..RLCA_MAX_BATCH) calls on `stream`; `calls` is host
 * memory, read before the function returns. */
rlca_status rlca_run_batch(const rlca_call *calls, int count, hipStream_t stream);

/* ------------------------------------------------- fused consumers of GAE
 * The summary's §9 (Discussion and Future Work) names fused loss operations
 * as the next step for the library; these two calls fuse the usual PPO
 * consumers of the advantages into the scan's epilogue and into one
 * streaming pass.  Each is one launch: every workgroup leaves one partial
 * sum in a caller-owned device workspace and takes a ticket from counters
 * at the workspace's start; the workgroup that takes the last ticket adds
 * the partials in a fixed order (reproducible bit for bit, whichever
 * workgroup is last), writes the result and sets the counters back to
 * zero.  The *_workspace_size call returns the workspace's size (0 for
 * an empty rollout or invalid sizes).  The workspace must be zero-filled
 * before its first use (one hipMemset, or a zero-filled allocation); every
 * call leaves it so, so it can be reused by later calls of either consumer
 * and any size up to its own.  A launch that did not run to completion
 * (a fault) may leave the counter set: zero the workspace again.  The
 * workspace is written like an output: calls that may run at the same time
 * need workspaces of their own.  workspace, stats and loss must be 8-byte
 * aligned; RLCA_ERR_INVALID_SIZE if workspace_bytes is too small;
 * RLCA_ERR_ALIASING if the workspace, stats or loss overlap any other array
 * of the call.  An empty rollout (num_envs * T == 0) writes nothing. */
size_t rlca_gae_stats_workspace_size(int64_t num_envs, int64_t T);

/* rlca_gae (fp32) that also reduces the advantages it computes: stats is
 * double[2] in device memory, {mean, sample standard deviation (divisor
 * N*T - 1; 0 when N*T == 1)} over all N*T steps, accumulated in fp64.  The
 * usual advantage normalization (A - mean) / (std + eps) needs exactly
 * these, without a second pass over the advantages.  advantages and returns
 * are bit for bit those of rlca_gae. */
rlca_status rlca_gae_stats(const float *rewards, const float *values, const uint8_t *terminated,
                           const uint8_t *truncated, const float *trunc_values,
                           const float *bootstrap, float gamma, float lambda, int64_t num_envs,
                           int64_t T, float *advantages, float *returns, double *stats,
                           void *workspace, size_t workspace_bytes, hipStream_t stream);

/* rlca_gae_stats for callers that cannot allocate (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc): the same
 * arguments without the workspace, the same kernels and the same results
 * bit for bit.  The ticket counter and partial sums live instead in a
 * buffer the library owns, RLCA_GAE_STATS_SCRATCH_BYTES of static device
 * memory that each GPU the library runs on holds until the process ends;
 * every size fits in it (the statistics launch never has more workgroups
 * than it has pairs), and a call that would need more returns
 * RLCA_ERR_INVALID_SIZE.  The call allocates nothing: the first call on
 * each device looks up the buffer's address there (hipGetSymbolAddress, no
 * allocation) and enqueues the zeroing of its counters on `stream`, one
 * small kernel (a caller that captures graphs should make that first call
 * before capturing); RLCA_ERR_HIP reports a failed lookup.  Every call on
 * one GPU shares its buffer and leaves its counters at zero: calls on one
 * stream are ordered and safe, but calls that may overlap on one GPU (on
 * different streams, or from threads that do not order them) race and
 * must use rlca_gae_stats with workspaces of their own. */
#define RLCA_GAE_STATS_SCRATCH_BYTES 69760
rlca_status rlca_gae_stats_noalloc(const float *rewards, const float *values,
                                   const uint8_t *terminated, const uint8_t *truncated,
                                   const float *trunc_values, const float *bootstrap, float gamma,
                                   float lambda, int64_t num_envs, int64_t T, float *advantages,
                                   float *returns, double *stats, hipStream_t stream);

size_t rlca_ppo_clip_loss_workspace_size(int64_t num_envs, int64_t T);

/* PPO clipped surrogate (Schulman et al. 2017, L^CLIP) as a loss, over the
 * M = num_envs * T steps of the [num_envs, T] arrays:
 *   A_hat_t = stats ? (A_t - stats[0]) / (stats[1] + norm_eps) : A_t
 *   rho_t   = exp(logp_new_t - logp_old_t)
 *   loss[0] = -(1/M) sum_t min(rho_t A_hat_t, clip(rho_t, 1-clip_eps, 1+clip_eps) A_hat_t)
 *   grad_logp_new[t] = d loss / d logp_new_t: -(1/M) rho_t A_hat_t where the
 *                      unclipped term is the smaller (ties included), else 0.
 * advantages, logp_new, logp_old [N,T] f32; stats double[2] as written by
 * rlca_gae_stats, nullable (no normalization); grad_logp_new [N,T] f32,
 * nullable; loss double[1] (device).  0 <= clip_eps < 1 and norm_eps >= 0,
 * finite, else RLCA_ERR_INVALID_VALUE.  Arithmetic per step is fp32, the
 * sums fp64. */
rlca_status rlca_ppo_clip_loss(const float *advantages, const double *stats,
                               const float *logp_new, const float *logp_old, float clip_eps,
                               float norm_eps, int64_t num_envs, int64_t T, float *grad_logp_new,
                               double *loss, void *workspace, size_t workspace_bytes,
                               hipStream_t stream);

/* ------------------------------------- operators of a recurrent policy or model
 * The forward affine recurrence as the core of a sequence model: a short
 * causal convolution and a selective state space scan over rows of T steps,
 * each with its gradients and its form for single steps, and the clipping of
 * the model's gradients by their global norm.
 *
 * Layout:   a row of T steps is contiguous in time, as everywhere in this
 *           header: activations are [num_seqs, channels, T] with free strides
 *           (in elements, not negative) between sequences and between
 *           channels, so a channel range of a projection's output
 *           [num_seqs, more channels, T] is read in place.  Outputs are
 *           dense; so are states and parameters.  Arrays must be aligned to
 *           their element size; speed, not results, depends on more.
 * Types:    `dtype` (RLCA_F32, RLCA_BF16 or RLCA_F16) is the storage type of
 *           the activations and of their gradients; arithmetic is fp32 and
 *           each output is rounded once.  Parameters, their gradients and the
 *           scan's states are float32 (a state is a running sum: rounding it
 *           to 16 bits at every step would lose what slow decays remember).
 *           The convolution's states are past inputs and have their type.
 * Episodes: `flags` [num_seqs, T] (nullable) marks episode boundaries inside
 *           the rows, under `convention` as for the forward scans above.  No
 *           state and no tap reaches across a start, not even a NaN or
 *           infinity; the state after the last step is 0 if that step's flag
 *           ends an episode (RLCA_RESET_AFTER_DONE).
 * Lengths:  `lengths` [num_seqs] int32 (nullable) gives each row's number of
 *           steps, in 0..T (values outside are taken as the nearer end).
 *           Steps past it change no state, get output and gradients 0, and
 *           what the inputs hold there is not used.
 * Sizes:    num_seqs * channels < 2^31 and T <= RLCA_MAX_T; a call with
 *           num_seqs, channels or T of 0 is a valid no-op where it has no
 *           state to hand on; with T = 0 the final state is the state, and
 *           the gradients of an empty sum are 0.  With channels = 0 nothing is
 *           launched or written: grad_B and grad_C, sums over no channels, are
 *           the caller's to clear.  A call whose launch would
 *           hold 2^32 threads is refused as too large: the scan over rows
 *           takes num_seqs * groups * ceil(channels / groups / 4) < 2^24, the
 *           convolution over rows channels < 2^24 (more if rows are short),
 *           the scan's step channels * states < 2^32.
 * Errors and memory: as stated at the top.  Workspaces need no
 *           initialisation, except rlca_clip_grad_norm's (as the fused
 *           consumers': zero-filled before its first use, and left so). */

/* The convolution:  pre_t = bias + sum_{k < width} weight[k] * x[t - (width-1) + k],
 * out_t = silu(pre_t) = pre_t / (1 + exp(-pre_t)), or pre_t with silu == 0.
 * Inputs before the row's first step are those of `state`, oldest first, or 0. */
typedef struct {
    int64_t num_seqs, channels, T;
    int32_t width;      /* taps: 2, 3 or 4 */
    int32_t silu;       /* nonzero: out = silu(pre) */
    int32_t dtype;      /* of x, out, state, grad_* of them */
    int32_t convention; /* rlca_reset_convention, for flags */
    const void *x;      /* [num_seqs, channels, T] */
    int64_t x_stride_seq, x_stride_channel;
    const float *weight;    /* [channels, width] */
    const float *bias;      /* [channels], nullable */
    const void *state;      /* [num_seqs, channels, width-1], nullable (=> 0) */
    const uint8_t *flags;   /* [num_seqs, T], nullable */
    const int32_t *lengths; /* [num_seqs], nullable */
    /* rlca_causal_conv */
    void *out;         /* [num_seqs, channels, T] */
    void *final_state; /* [num_seqs, channels, width-1], nullable: the state for the next row */
    /* rlca_causal_conv_backward */
    const void *grad_out; /* [num_seqs, channels, T] */
    int64_t grad_stride_seq, grad_stride_channel;
    const void *grad_final_state; /* [num_seqs, channels, width-1], nullable (=> 0) */
    void *grad_x;                 /* [num_seqs, channels, T] */
    float *grad_weight;           /* [channels, width] */
    float *grad_bias;             /* [channels], nullable */
    void *grad_state;             /* [num_seqs, channels, width-1], nullable */
} rlca_conv_call;

rlca_status rlca_causal_conv(const rlca_conv_call *call, hipStream_t stream);

/* The gradients of the call whose inputs `call` holds: pre is computed again
 * from x.  Sums over sequences and steps run in a fixed order (reproducible
 * bit for bit).  The workspace holds each row's partial sums. */
size_t rlca_causal_conv_backward_workspace_size(const rlca_conv_call *call);
rlca_status rlca_causal_conv_backward(const rlca_conv_call *call, void *workspace,
                                      size_t workspace_bytes, hipStream_t stream);

/* The scan, for each channel d with `states` running values:
 *   dt_t = softplus(delta_t + delta_bias), or delta_t + delta_bias with softplus == 0
 *   h_t  = exp(dt_t A) h_{t-1} + dt_t u_t B_t        (h: [states]; h_{t-1} = 0 at a start)
 *   y_t  = (sum_s C_t[s] h_t[s] + D u_t) * silu(z_t)   (the gate only where z is given)
 * B and C are shared by the channels / groups consecutive channels of a group.
 * States may grow (A above 0, or dt below 0 without softplus): they are what the
 * recurrence gives step by step, however large the product of many decays, and
 * strongly growing rows take up to three times as long. */
#define RLCA_MAX_STATES 128

typedef struct {
    int64_t num_seqs, channels, T;
    int32_t states;   /* 1 .. RLCA_MAX_STATES */
    int32_t groups;   /* divides channels */
    int32_t softplus; /* nonzero: dt = softplus(...) */
    int32_t dtype;    /* of u, delta, B, C, z, y and of their gradients */
    int32_t convention;
    const void *u, *delta; /* [num_seqs, channels, T] */
    int64_t u_stride_seq, u_stride_channel, delta_stride_seq, delta_stride_channel;
    const float *A;    /* [channels, states]; below 0 for a decaying state */
    const void *B, *C; /* [num_seqs, groups, states, T] */
    int64_t B_stride_seq, B_stride_group, B_stride_state;
    int64_t C_stride_seq, C_stride_group, C_stride_state;
    const float *D;          /* [channels], nullable (=> 0) */
    const float *delta_bias; /* [channels], nullable (=> 0) */
    const void *z;           /* [num_seqs, channels, T], nullable: no gate */
    int64_t z_stride_seq, z_stride_channel;
    const float *state;     /* [num_seqs, channels, states], nullable (=> 0) */
    const uint8_t *flags;   /* [num_seqs, T], nullable */
    const int32_t *lengths; /* [num_seqs], nullable */
    /* rlca_selective_scan.  checkpoints (nullable) is what the backward call
     * needs of the forward one: states at fixed steps, laid out for it. */
    void *y;            /* [num_seqs, channels, T] */
    float *final_state; /* [num_seqs, channels, states], nullable */
    float *checkpoints; /* rlca_selective_scan_checkpoints_size bytes */
    /* rlca_selective_scan_backward (reads checkpoints) */
    const void *grad_y; /* [num_seqs, channels, T] */
    int64_t grad_stride_seq, grad_stride_channel;
    const float *grad_final_state; /* [num_seqs, channels, states], nullable (=> 0) */
    void *grad_u, *grad_delta;     /* [num_seqs, channels, T] */
    float *grad_A;                 /* [channels, states] */
    void *grad_B, *grad_C;         /* [num_seqs, groups, states, T] */
    float *grad_D, *grad_delta_bias; /* [channels], nullable */
    void *grad_z;                    /* [num_seqs, channels, T]; required iff z */
    float *grad_state;               /* [num_seqs, channels, states], nullable */
} rlca_scan_call;

size_t rlca_selective_scan_checkpoints_size(const rlca_scan_call *call);
rlca_status rlca_selective_scan(const rlca_scan_call *call, hipStream_t stream);

/* The gradients of the call whose inputs and checkpoints `call` holds.
 * Nothing is accumulated into what the outputs held before, and all sums run
 * in a fixed order (reproducible bit for bit).  Sums over the channels of a
 * group, over sequences and over steps are float32 or wider. */
size_t rlca_selective_scan_backward_workspace_size(const rlca_scan_call *call);
rlca_status rlca_selective_scan_backward(const rlca_scan_call *call, void *workspace,
                                         size_t workspace_bytes, hipStream_t stream);

/* One step of the convolution and of the scan for each of `num_seqs`
 * sequences (a generated token, an environment's next action).  Sequence n's
 * state is place slots[n] of a pool of `places` states (slots == NULL: place
 * n, and places >= num_seqs), read and rewritten in place.  A slot outside
 * 0..places-1 is an empty seat of the batch: its output is 0 and no state is
 * touched.  The slots of one call must differ (two sequences would race on
 * one state).  starts [num_seqs] (nullable): nonzero begins an episode with
 * this step, so the state is taken as 0. */
typedef struct {
    int64_t num_seqs, channels, places;
    int32_t width, silu, dtype;
    const void *x; /* [num_seqs, channels], rows x_stride_seq elements apart */
    int64_t x_stride_seq;
    const float *weight, *bias;
    void *state;           /* [places, channels, width-1], in and out */
    const int32_t *slots;  /* [num_seqs], nullable */
    const uint8_t *starts; /* [num_seqs], nullable */
    void *out;             /* [num_seqs, channels] */
} rlca_conv_step_call;

rlca_status rlca_causal_conv_step(const rlca_conv_step_call *call, hipStream_t stream);

typedef struct {
    int64_t num_seqs, channels, places;
    int32_t states, groups, softplus, dtype;
    const void *u, *delta; /* [num_seqs, channels] */
    int64_t u_stride_seq, delta_stride_seq;
    const float *A;
    const void *B, *C; /* [num_seqs, groups, states] */
    int64_t B_stride_seq, B_stride_group, C_stride_seq, C_stride_group;
    const float *D, *delta_bias;
    const void *z; /* [num_seqs, channels], nullable */
    int64_t z_stride_seq;
    float *state; /* [places, channels, states], in and out */
    const int32_t *slots;
    const uint8_t *starts;
    void *y; /* [num_seqs, channels] */
} rlca_scan_step_call;

rlca_status rlca_selective_step(const rlca_scan_step_call *call, hipStream_t stream);

/* The global norm of a model's gradients, and the gradients scaled to at most
 * max_norm:
 *   norm[0] = sqrt(sum over all tensors of x^2)      (double; squares and sums in fp64)
 *   out = x * min(1, max_norm / (norm[0] + eps))
 * (and out = x where the norm is 0).  out may be data itself (in place, the
 * usual case) or another array that overlaps no array of the call.  With
 * max_norm = +infinity only the norm is computed, and out is not used.  A NaN
 * gradient makes the norm and every scaled value NaN, as the formula says; with
 * an infinite one the scale is 0 and infinite values become NaN.  max_norm >= 0, eps >= 0 and finite.  `tensors` is host memory,
 * read before the function returns; tensors of count 0 are skipped, and with
 * nothing to sum the norm is 0.  The sums run in a fixed order: the norm is
 * reproducible bit for bit. */
typedef struct {
    const void *data;
    void *out;
    int64_t count;
    int32_t dtype;
} rlca_grad_tensor;

#define RLCA_CLIP_WORKSPACE_BYTES 20736
rlca_status rlca_clip_grad_norm(const rlca_grad_tensor *tensors, int64_t num_tensors,
                                double max_norm, double eps, double *norm, void *workspace,
                                size_t workspace_bytes, hipStream_t stream);

/* ------------------------------------------- operators of a block and of a search
 * What stands around the recurrences in a residual stack of blocks, and in
 * generating with it, over the same rows and pools: the gated linear recurrence
 * with its gradients and its single step, the root-mean-square norm with the
 * residual's addition, and a beam search's selection and reordering of states.
 * Layout, types, episodes, lengths, sizes, errors and memory are as above.
 *
 * The gated recurrence: one state a channel, whose decay and input are gated
 * step by step,
 *   r_t = sigmoid(decay_gate_t + decay_bias),  i_t = sigmoid(input_gate_t + input_bias),
 *   L_t = scale softplus(decay) r_t,  a_t = exp(-L_t),
 *   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) i_t x_t      (h_{t-1} = 0 at a start);
 * out_t is h_t, rounded once.  A state decays at every step and cannot grow; a_t is
 * float32, so steps with L_t below 1e-7 do not decay.  An infinite state does not stay
 * infinity for certain: where a run's decays multiply to less than float32 holds, 0
 * times it is NaN.  Either stays, in the states and back through the gradients, until
 * an episode starts.  The checkpoints (nullable)
 * are the states that the backward call starts from.  scale is within 1e-30 ..
 * 1e30, channels below 2^25.  The workspaces need no initialisation; the forward
 * call's may be of size 0. */
typedef struct {
    int64_t num_seqs, channels, T;
    int32_t dtype;      /* of x, the gates, out and their gradients */
    int32_t convention; /* rlca_reset_convention, for flags */
    double scale;
    const void *x, *input_gate, *decay_gate; /* [num_seqs, channels, T] */
    int64_t x_stride_seq, x_stride_channel;
    int64_t input_stride_seq, input_stride_channel;
    int64_t decay_stride_seq, decay_stride_channel;
    const float *decay;                   /* [channels] */
    const float *input_bias, *decay_bias; /* [channels], nullable (=> 0) */
    const float *state;                   /* [num_seqs, channels], nullable (=> 0) */
    const uint8_t *flags;                 /* [num_seqs, T], nullable */
    const int32_t *lengths;               /* [num_seqs], nullable */
    /* rlca_gated_recurrence */
    void *out;          /* [num_seqs, channels, T] */
    float *final_state; /* [num_seqs, channels], nullable */
    float *checkpoints; /* rlca_gated_recurrence_checkpoints_size bytes, nullable */
    /* rlca_gated_recurrence_backward (reads checkpoints) */
    const void *grad_out; /* [num_seqs, channels, T] */
    int64_t grad_stride_seq, grad_stride_channel;
    const float *grad_final_state; /* [num_seqs, channels], nullable (=> 0) */
    void *grad_x, *grad_input_gate, *grad_decay_gate; /* [num_seqs, channels, T] */
    float *grad_decay;                                /* [channels] */
    float *grad_input_bias, *grad_decay_bias;         /* [channels], nullable */
    float *grad_state;                                /* [num_seqs, channels], nullable */
} rlca_gated_call;

size_t rlca_gated_recurrence_checkpoints_size(const rlca_gated_call *call);
size_t rlca_gated_recurrence_workspace_size(const rlca_gated_call *call);
rlca_status rlca_gated_recurrence(const rlca_gated_call *call, void *workspace,
                                  size_t workspace_bytes, hipStream_t stream);

/* The gradients of the call whose inputs and checkpoints `call` holds.  Nothing is
 * accumulated into what the outputs held before, and all sums run in a fixed order
 * (reproducible bit for bit). */
size_t rlca_gated_recurrence_backward_workspace_size(const rlca_gated_call *call);
rlca_status rlca_gated_recurrence_backward(const rlca_gated_call *call, void *workspace,
                                           size_t workspace_bytes, hipStream_t stream);

/* One step for each of `num_seqs` sequences, with a pool of states, slots and starts
 * as for rlca_selective_step. */
typedef struct {
    int64_t num_seqs, channels, places;
    int32_t dtype;
    double scale;
    const void *x, *input_gate, *decay_gate; /* [num_seqs, channels] */
    int64_t x_stride_seq, input_stride_seq, decay_stride_seq;
    const float *decay, *input_bias, *decay_bias;
    float *state; /* [places, channels], in and out */
    const int32_t *slots;
    const uint8_t *starts;
    void *out; /* [num_seqs, channels] */
} rlca_gated_step_call;

rlca_status rlca_gated_step(const rlca_gated_step_call *call, hipStream_t stream);

/* The root-mean-square norm over the channels of each step, after a residual's
 * addition:
 *   s = x + residual (rounded to the storage type; s = x without a residual),
 *   y = s / sqrt(mean over channels of s^2 + eps) * weight.
 * s is the residual stream that goes on, and it is normed as it is stored.  The
 * output is y in the storage type, or in 8 bits (OCP e4m3) with one float32 scale a
 * step: scale = max(max over channels of |y| / 448, 2^-120), out8 = y / scale rounded
 * to nearest even.  Squares and sums are float32, and are scaled down where they would
 * overflow.  Steps past a row's length get output, sum, scale and gradient 0; with no
 * channels all scales are 0.  T = 1 with x_stride_channel = 1 (and the residual's and
 * gradients' too) is the norm of dense rows of channels: a generated token's, or any
 * [tokens, channels] array's.  Their 8-bit output is what an 8-bit matrix product takes
 * as it is; in rows over time a step's channels lie T apart, and a product that wants
 * them side by side takes a transposed copy.  eps is within 1e-30 .. 1e30. */
typedef struct {
    int64_t num_seqs, channels, T;
    int32_t dtype;
    double eps;
    const void *x; /* [num_seqs, channels, T] */
    int64_t x_stride_seq, x_stride_channel;
    const void *residual; /* [num_seqs, channels, T], nullable */
    int64_t residual_stride_seq, residual_stride_channel;
    const float *weight;    /* [channels], nullable (=> 1) */
    const int32_t *lengths; /* [num_seqs], nullable */
    /* rlca_rms_norm */
    void *out;    /* [num_seqs, channels, T]; NULL where out8 is wanted */
    uint8_t *out8; /* [num_seqs, channels, T]; NULL where out is */
    float *scale; /* [num_seqs, T]; required iff out8 */
    void *sum;    /* [num_seqs, channels, T]; required iff residual */
    /* rlca_rms_norm_backward: x is what was normed (s), residual is not used */
    const void *grad_out; /* [num_seqs, channels, T] */
    int64_t grad_stride_seq, grad_stride_channel;
    const void *grad_sum; /* [num_seqs, channels, T], nullable: added to grad_x */
    int64_t grad_sum_stride_seq, grad_sum_stride_channel;
    void *grad_x;       /* [num_seqs, channels, T]: the gradient of s, so of x and residual */
    float *grad_weight; /* [channels], nullable */
} rlca_norm_call;

rlca_status rlca_rms_norm(const rlca_norm_call *call, hipStream_t stream);

/* The gradients: the workspace needs no initialisation, and all sums run in a fixed
 * order (reproducible bit for bit). */
size_t rlca_rms_norm_backward_workspace_size(const rlca_norm_call *call);
rlca_status rlca_rms_norm_backward(const rlca_norm_call *call, void *workspace,
                                   size_t workspace_bytes, hipStream_t stream);

/* A beam search's selection.  For each of num_searches searches, over all `beams`
 * beams and `vocab` tokens, the `picks` candidates with the highest
 *   total = score_b + (logit_bv - log sum_v exp(logit_bv)),
 * best first, equal ones by beam (the lower first), those of one beam by logit and then
 * token (the lower first).  Exponentials are float32, their sums over a beam and the
 * totals float64: totals are good to 2e-6 and usually to 1e-7, and they are compared
 * before the one rounding to float32.  A beam that is finished has one candidate, pad_token
 * at its own score; its other totals are -infinity.  So are all totals of a beam
 * whose score is -infinity (an unused one: its logits do not count, whatever they
 * hold) and those of logits of -infinity (tokens that are not allowed; all of them
 * may be).  A NaN or +infinity among a beam's logits, or as its score, makes its
 * totals NaN, and NaN ranks first.  beams and picks are 1 .. RLCA_MAX_BEAMS, picks at
 * most beams * vocab, beams * vocab < 2^31, and num_searches * beams *
 * ceil(vocab / 2048) < 2^24. */
#define RLCA_MAX_BEAMS 64

typedef struct {
    int64_t num_searches, beams, vocab;
    int32_t picks, dtype, pad_token;
    const void *logits; /* [num_searches, beams, vocab] */
    int64_t logits_stride_search, logits_stride_beam;
    const float *scores;     /* [num_searches, beams] */
    const uint8_t *finished; /* [num_searches, beams], nullable */
    float *out_scores;       /* [num_searches, picks] */
    int32_t *out_tokens, *out_parents; /* [num_searches, picks] */
} rlca_beam_call;

size_t rlca_beam_select_workspace_size(const rlca_beam_call *call);
rlca_status rlca_beam_select(const rlca_beam_call *call, void *workspace, size_t workspace_bytes,
                             hipStream_t stream);

/* The beams' states after a selection, in any number of pools [places, ...] of
 * place_bytes a place.  Beam k of a search goes on from the state of its beam
 * parents[k]: the first child of a parent keeps the parent's place, and each other
 * one gets the place of a beam without children (both in order), to which the state
 * is copied in every pool.  new_slots is where each beam's state is then; no other
 * place is written.  Slots as for the single steps: those of one call must differ,
 * and one outside 0..places-1 holds no state (nothing is copied from or to it).  A
 * parent outside 0..beams-1 makes an unused beam, which gets a free place and no
 * state.  `pools` is host memory, read before the function returns; beams <=
 * RLCA_MAX_BEAMS. */
typedef struct {
    void *data;
    int64_t place_bytes;
} rlca_state_pool;

rlca_status rlca_beam_reorder(const rlca_state_pool *pools, int64_t num_pools,
                              int64_t num_searches, int64_t beams, int64_t places,
                              const int32_t *slots, const int32_t *parents, int32_t *new_slots,
                              hipStream_t stream);

/* Static description of a status code (never NULL). */
const char *rlca_status_string(rlca_status status);

#ifdef __cplusplus
}
#endif

#endif /* RLCA_H */
