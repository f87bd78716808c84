"""A decode loop with speculation in which nothing leaves the GPU between steps.

One layer of a random model stands for the target; what matters is the order of
the calls of a step, all of them on one stream and, after the first step, in one
CUDA graph:

    kv_block_step        blocks and slots, from the last step's accepted lengths
    kv_append            the new tokens' keys and values, 8 bits a value
    spec_attention       the new tokens' queries over the cache
    spec_process_logits  penalties of what the request has made, and its grammar
    spec_verify          which drafts stand, and the token after them

Run: python examples/decode_step.py [requests] [steps]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_verification_80_gb300 as sd  # noqa: E402


class Decoder:
    """State of B requests; `allowed` [B, V] (bool) is each one's grammar."""

    def __init__(self, B, drafts=4, V=4096, hidden=512, Hq=16, H=4, D=64, block_size=16, max_len=512, allowed=None,
                 seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
        i32 = lambda *s, fill=0: torch.full(s, fill, dtype=torch.int32, device="cuda")  # noqa: E731
        self.B, self.n, self.V, self.Hq, self.H, self.D, self.max_len = B, drafts, V, Hq, H, D, max_len
        self.block_size = block_size
        self.embed, self.position = rand(V, hidden), 0.3 * rand(max_len + drafts + 1, hidden)
        self.w_qkv, self.w_out, self.w_head = (rand(hidden, (Hq + 2 * H) * D) / hidden ** 0.5,
                                               rand(Hq * D, hidden) / (Hq * D) ** 0.5, rand(V, hidden) / hidden ** 0.5)
        width = (max_len + drafts + block_size) // block_size
        blocks = B * width
        self.k_cache, self.v_cache = (torch.zeros(blocks, H, block_size, D, dtype=torch.uint8, device="cuda").view(
            torch.float8_e4m3fn) for _ in range(2))
        self.k_scale, self.v_scale = (torch.zeros(blocks, H, device="cuda") for _ in range(2))
        self.table, self.ring = i32(B, width), torch.arange(blocks, dtype=torch.int32, device="cuda")
        # the state that a step reads and leaves for the next
        T = B * (drafts + 1)
        self.state = sd.BlockStep(kv_len=i32(B), held=i32(B), ring_state=torch.tensor([0, blocks], dtype=torch.int32, device="cuda"),
                                  cu_tokens=i32(B + 1), cu_blocks=i32(B + 1), slot_map=i32(T), positions=i32(T))
        self.accepted, self.last = i32(B), i32(B)
        self.history, self.history_len, self.prompt_len = i32(B, max_len), i32(B), i32(B)
        self.new_tokens, self.draft_len = i32(B, fill=drafts + 1), i32(B, fill=drafts)
        self.temperature = torch.zeros(B, device="cuda")
        self.repetition = torch.full((B,), 1.1, device="cuda")
        self.frequency = torch.full((B,), 0.2, device="cuda")
        self.mask = self.mask_rows = None
        if allowed is not None:
            bits = torch.nn.functional.pad(allowed, (0, -V % 32)).view(B, -1, 32).long()
            words = (bits << torch.arange(32, device="cuda")).sum(2)
            self.mask = torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)
            self.mask_rows = torch.arange(B, dtype=torch.int32, device="cuda").repeat_interleave(drafts + 1).view(B, -1)
        self.attention_workspace = sd.new_attention_workspace()
        self.verify_workspace = sd.new_workspace(B, drafts, V)
        self.error = i32(1)
        self.graph = None

    def _layer(self, tokens, blocks):
        """The new tokens' hidden states after the layer."""
        T = tokens.numel()
        x = self.embed[tokens] + self.position[blocks.positions.clamp(min=0)]
        qkv = (x @ self.w_qkv).view(T, self.Hq + 2 * self.H, self.D)
        q, k, v = qkv.split((self.Hq, self.H, self.H), 1)
        sd.kv_append(k, v, blocks.slot_map, self.k_cache, self.v_cache, self.k_scale, self.v_scale)
        o = sd.spec_attention(q, blocks.cu_tokens, blocks.kv_len, self.table, self.k_cache, self.v_cache, self.k_scale,
                              self.v_scale, workspace=self.attention_workspace)
        return x + o.view(T, -1) @ self.w_out

    def prompt(self, tokens):
        """The requests' prompts [B, P]; one token is made."""
        B, P = tokens.shape
        blocks = sd.kv_block_step(self.table, self.state.kv_len, self.state.held, torch.full_like(self.accepted, P),
                                  self.ring, self.state.ring_state, self.block_size, B * P, error_word=self.error)
        for name in ("kv_len", "held", "ring_state"):
            getattr(self.state, name).copy_(getattr(blocks, name))
        x = self._layer(tokens.reshape(-1), blocks)
        self.history[:, :P] = tokens
        self.prompt_len.fill_(P)
        self.history_len.fill_(P)
        logits = (x.view(B, P, -1)[:, -1:] @ self.w_head.t()).contiguous()
        first = None if self.mask_rows is None else self.mask_rows[:, :1].contiguous()
        sd.spec_process_logits(logits, self.history, self.prompt_len, self.history_len, repetition=self.repetition,
                               frequency=self.frequency, mask=self.mask, mask_rows=first, error_word=self.error)
        self.last.copy_(logits.view(B, -1).argmax(1))
        self.history[:, P] = self.last
        self.history_len.add_(1)
        self.accepted.fill_(P - 1)  # all of the prompt stays

    def _step(self):
        B, n = self.B, self.n
        # drafts: the head on the embedding alone
        fed = [self.last]
        for _ in range(n):
            fed.append((self.embed[fed[-1]] @ self.w_head.t()).argmax(1).to(torch.int32))
        fed = torch.stack(fed, 1)
        drafts = fed[:, 1:].contiguous()
        s = sd.kv_block_step(self.table, self.state.kv_len, self.state.held, self.new_tokens, self.ring, self.state.ring_state,
                             self.block_size, B * (n + 1), accepted_len=self.accepted, out=self.state, error_word=self.error)
        x = self._layer(fed.view(-1), s)
        logits = (x @ self.w_head.t()).view(B, n + 1, self.V)
        sd.spec_process_logits(logits, self.history, self.prompt_len, self.history_len, draft_tokens=drafts,
                               draft_len=self.draft_len, repetition=self.repetition, frequency=self.frequency,
                               mask=self.mask, mask_rows=self.mask_rows, error_word=self.error)
        _, out = sd.spec_verify(logits, None, drafts, self.draft_len, self.temperature, accepted_len=self.accepted,
                                workspace=self.verify_workspace)
        # the accepted drafts and the token after them are the request's
        j = torch.arange(n + 1, device="cuda")
        at = self.history_len[:, None] + j
        made = (j <= self.accepted[:, None]) & (at < self.max_len)
        at = at.clamp(max=self.max_len - 1).long()
        self.history.scatter_(1, at, torch.where(made, out, self.history.gather(1, at)))
        self.history_len.add_(self.accepted + 1).clamp_(max=self.max_len)
        self.last.copy_(out.gather(1, self.accepted[:, None].long()).view(-1))

    def step(self):
        """A verify step of all requests: up to n + 1 tokens each."""
        if self.graph is None:
            self._step()  # (the first also allocates what the graph must not)
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self._step()
        else:
            self.graph.replay()


def main(B=64, steps=20):
    g = torch.Generator(device="cuda").manual_seed(1)
    allowed = torch.rand(B, 4096, generator=g, device="cuda") < 0.5
    d = Decoder(B, allowed=allowed)
    d.prompt(torch.randint(0, d.V, (B, 100), generator=g, device="cuda", dtype=torch.int32))
    d.step()
    d.step()
    before = int(d.history_len.sum())
    t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    t0.record()
    for _ in range(steps):
        d.step()
    t1.record()
    torch.cuda.synchronize()
    made = int(d.history_len.sum()) - before
    print(f"{B} requests, {steps} steps: {made / steps / B:.2f} tokens a request and step, "
          f"{t0.elapsed_time(t1) * 1000 / steps:.0f} us a step, error word {int(d.error)}")
    print("request 0 made", d.history[0, 100:int(d.history_len[0])].tolist())


if __name__ == "__main__":
    main(*(int(x) for x in sys.argv[1:]))
